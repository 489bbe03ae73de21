// Attention of trees for head_dim 256 over a bf16 cache.
#include "attn_tree.cuh"

namespace attn {
cudaError_t launch_tree_hd256_bf16(const TreeRequest &r) { return launch_tree_for<256, __nv_bfloat16>(r); }
} // namespace attn
