// Paged decode kernels for head_dim 128 over a e4m3 cache.
#include "attn_paged_impl.cuh"

namespace attn {
cudaError_t launch_paged_hd128_e4m3(const PagedRequest &r) { return launch_paged_for<128, E4m3>(r); }
} // namespace attn
