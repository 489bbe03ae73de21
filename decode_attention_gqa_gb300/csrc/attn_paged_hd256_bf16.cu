// Paged decode kernels for head_dim 256 over a bf16 cache.
#include "attn_paged_impl.cuh"

namespace attn {
cudaError_t launch_paged_hd256_bf16(const PagedRequest &r) { return launch_paged_for<256, __nv_bfloat16>(r); }
} // namespace attn
