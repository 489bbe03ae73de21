// Attention of trees for head_dim 64 over a bf16 cache.
#include "attn_tree.cuh"

namespace attn {
cudaError_t launch_tree_hd64_bf16(const TreeRequest &r) { return launch_tree_for<64, __nv_bfloat16>(r); }
} // namespace attn
