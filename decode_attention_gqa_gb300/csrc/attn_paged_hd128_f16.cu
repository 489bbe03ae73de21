// Paged decode kernels for head_dim 128 over a f16 cache.
#include "attn_paged_impl.cuh"

namespace attn {
cudaError_t launch_paged_hd128_f16(const PagedRequest &r) { return launch_paged_for<128, __half>(r); }
} // namespace attn
