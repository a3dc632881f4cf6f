// The tensor-core attention for head dim 64.
#include "tree_attn_tc.cuh"

namespace dspark {
namespace attn {
DSPARK_ATTN_TC_DEFINE(64)
}
}  // namespace dspark
