// Attention of trees for head_dim 256 over a f16 cache.
#include "attn_tree.cuh"

namespace attn {
cudaError_t launch_tree_hd256_f16(const TreeRequest &r) { return launch_tree_for<256, __half>(r); }
} // namespace attn
