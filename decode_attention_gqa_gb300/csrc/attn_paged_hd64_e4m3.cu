// Paged decode kernels for head_dim 64 over a e4m3 cache.
#include "attn_paged_impl.cuh"

namespace attn {
cudaError_t launch_paged_hd64_e4m3(const PagedRequest &r) { return launch_paged_for<64, E4m3>(r); }
} // namespace attn
