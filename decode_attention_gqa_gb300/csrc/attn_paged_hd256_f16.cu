// Paged decode kernels for head_dim 256 over a f16 cache.
#include "attn_paged_impl.cuh"

namespace attn {
cudaError_t launch_paged_hd256_f16(const PagedRequest &r) { return launch_paged_for<256, __half>(r); }
} // namespace attn
