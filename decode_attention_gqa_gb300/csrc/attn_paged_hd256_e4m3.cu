// Paged decode kernels for head_dim 256 over a e4m3 cache.
#include "attn_paged_impl.cuh"

namespace attn {
cudaError_t launch_paged_hd256_e4m3(const PagedRequest &r) { return launch_paged_for<256, E4m3>(r); }
} // namespace attn
