// The tensor-core attention for head dim 128.
#include "tree_attn_tc.cuh"

namespace dspark {
namespace attn {
DSPARK_ATTN_TC_DEFINE(128)
}
}  // namespace dspark
