// Which kernel serves a call of the drafted tokens' attention.
#include <cstdlib>
#include <cstring>

#include "tree_attn_tc.cuh"

namespace dspark {
namespace attn {
DSPARK_ATTN_DECLARE(64)
DSPARK_ATTN_DECLARE(128)
DSPARK_ATTN_DECLARE(256)
DSPARK_ATTN_TC_DECLARE(64)
DSPARK_ATTN_TC_DECLARE(128)
}  // namespace attn

namespace {

// The tensor-core kernel takes head dims 64 and 128 where the mean request
// has more than kTcRows query rows per KV head.  DSPARK_TREE_ATTN_KERNEL=mma
// or =tc pins one (tc: for the head dims it has) for the calls made while it
// is set; the tests run both.
constexpr int64_t kTcRows = 32;

bool use_tc(int64_t rows, int group, int requests, int head_dim)
{
    if (head_dim > 128)
        return false;
    const char *e = std::getenv("DSPARK_TREE_ATTN_KERNEL");
    if (e && std::strcmp(e, "mma") == 0)
        return false;
    if (e && std::strcmp(e, "tc") == 0)
        return true;
    return rows * group > kTcRows * requests;
}

}  // namespace

int64_t tree_attention_workspace(int64_t rows, int num_heads, int num_kv_heads, int head_dim, int requests, bool fp8,
                                 cudaError_t &e)
{
    if (use_tc(rows, num_heads / num_kv_heads, requests, head_dim))
        return head_dim == 64 ? attn::workspace_tc<64>(fp8, e) : attn::workspace_tc<128>(fp8, e);
    const int wr = attn::row_warps(rows, num_heads / num_kv_heads, requests);
    switch (head_dim) {
    case 64: return attn::workspace_d<64>(wr, fp8, e);
    case 128: return attn::workspace_d<128>(wr, fp8, e);
    default: return attn::workspace_d<256>(wr, fp8, e);
    }
}

cudaError_t launch_tree_attention(const AttnParams &p, int head_dim, bool fp8, cudaStream_t stream)
{
    if (use_tc(p.num_rows, p.group, p.num_requests, head_dim))
        return head_dim == 64 ? attn::attention_tc_d<64>(p, fp8, stream) : attn::attention_tc_d<128>(p, fp8, stream);
    const int wr = attn::row_warps(p.num_rows, p.group, p.num_requests);
    switch (head_dim) {
    case 64: return attn::attention_d<64>(p, wr, fp8, stream);
    case 128: return attn::attention_d<128>(p, wr, fp8, stream);
    default: return attn::attention_d<256>(p, wr, fp8, stream);
    }
}

}  // namespace dspark
