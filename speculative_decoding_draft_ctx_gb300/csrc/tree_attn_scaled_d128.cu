// The drafted tokens' attention (mma.sync) over page-scaled caches for head dim 128
// (one translation unit per head dim, so that they compile side by side).
#include "tree_attn_split.cuh"

namespace dspark {
namespace attn {
DSPARK_ATTN_SCALED_DEFINE(128)
}
}  // namespace dspark
