// Attention of trees for head_dim 64 over a f16 cache.
#include "attn_tree.cuh"

namespace attn {
cudaError_t launch_tree_hd64_f16(const TreeRequest &r) { return launch_tree_for<64, __half>(r); }
} // namespace attn
