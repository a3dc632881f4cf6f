// The drafted tokens' attention (mma.sync) for head dim 256
// (one translation unit per head dim, so that they compile side by side).
#include "tree_attn_mma.cuh"

namespace dspark {
namespace attn {
DSPARK_ATTN_DEFINE(256)
}
}  // namespace dspark
