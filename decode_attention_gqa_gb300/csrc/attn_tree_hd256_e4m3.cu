// Attention of trees for head_dim 256 over a e4m3 cache.
#include "attn_tree.cuh"

namespace attn {
cudaError_t launch_tree_hd256_e4m3(const TreeRequest &r) { return launch_tree_for<256, E4m3>(r); }
} // namespace attn
