// The drafted tokens' attention (tcgen05) over page-scaled caches for head dim 64
// (one translation unit per head dim, so that they compile side by side).
#include "tree_attn_tc.cuh"

namespace dspark {
namespace attn {
DSPARK_ATTN_TC_SCALED_DEFINE(64)
}
}  // namespace dspark
