// Which kernel serves a call of the drafted tokens' attention and of the
// weight accumulation.
#include "tree_attn_mma.cuh"

namespace dspark {
namespace attn {
DSPARK_ATTN_DECLARE(64)
DSPARK_ATTN_DECLARE(128)
DSPARK_ATTN_DECLARE(256)
}  // namespace attn

int64_t tree_attention_workspace(int64_t rows, int num_heads, int num_kv_heads, int head_dim, int requests, bool fp8,
                                 cudaError_t &e)
{
    const int wr = attn::row_warps(rows, num_heads / num_kv_heads, requests);
    switch (head_dim) {
    case 64: return attn::workspace_d<64>(wr, fp8, e);
    case 128: return attn::workspace_d<128>(wr, fp8, e);
    default: return attn::workspace_d<256>(wr, fp8, e);
    }
}

cudaError_t launch_tree_attention(const AttnParams &p, int head_dim, bool fp8, cudaStream_t stream)
{
    const int wr = attn::row_warps(p.num_rows, p.group, p.num_requests);
    switch (head_dim) {
    case 64: return attn::attention_d<64>(p, wr, fp8, stream);
    case 128: return attn::attention_d<128>(p, wr, fp8, stream);
    default: return attn::attention_d<256>(p, wr, fp8, stream);
    }
}

cudaError_t launch_attention_weight(const AttnParams &p, int head_dim, bool fp8, cudaStream_t stream)
{
    switch (head_dim) {
    case 64: return attn::weight_d<64>(p, fp8, stream);
    case 128: return attn::weight_d<128>(p, fp8, stream);
    default: return attn::weight_d<256>(p, fp8, stream);
    }
}

}  // namespace dspark
