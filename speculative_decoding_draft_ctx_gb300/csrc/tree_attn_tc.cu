// The tensor-core attention for head dims 64 and 128.
#include "tree_attn_tc.cuh"

namespace dspark {
namespace attn {
DSPARK_ATTN_TC_DEFINE(64)
DSPARK_ATTN_TC_DEFINE(128)
}  // namespace attn
}  // namespace dspark
