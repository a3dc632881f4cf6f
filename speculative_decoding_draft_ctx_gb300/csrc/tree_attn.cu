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
// has more than kTcRows query rows per KV head and the block table has room
// for more than one tile of 128 keys per two SMs (lengths are on the device:
// the room is what the host knows).  Measured, D 128, mma.sync against it, us:
//   rows 32, 8 requests x 8 heads over 4,000 tokens   37 / 39, fp8 32 / 45
//   rows 56, 16 x 8 over 8,000                        135 / 102, fp8 142 / 129
//   rows 504, 1 x 4 over 16,000                       70 / 39, fp8 74 / 44
//   rows 56, 1 x 8 over 500 (32 tiles)                11.9 / 12.6, fp8 13.0 / 14.5
//   rows 56, 1 x 8 over 2,000 (128 tiles)             18.2 / 18.3, fp8 18.7 / 19.5
//   rows 504, 1 x 4 over 2,000 (68 tiles)             23.7 / 29.6, fp8 24.6 / 28.9
//   rows 56, 64 x 8 over 1,024 to 8,192               233 / 194, fp8 246 / 246
//   the same at D 64                                  166 / 160, fp8 155 / 233
// The last figure is the rule's one loss among these: head dim 64 over fp8.  It
// also loses where the mean says little: 63 single tokens over 2,000 and a tree
// of 64 over 131,072 (group 8) run in items of 16 rows, 2,485 / 438, fp8 2,123
// / 473; rows of the largest request would have to come from the caller.
// DSPARK_TREE_ATTN_KERNEL=mma or =tc pins one (tc: for the head dims it has)
// for the calls made while it is set; the tests run both.
constexpr int64_t kTcRows = 32;

enum Pin { kNone, kMma, kTc };

Pin pinned(int head_dim)
{
    if (head_dim > 128)
        return kMma;
    const char *e = std::getenv("DSPARK_TREE_ATTN_KERNEL");
    return !e ? kNone : std::strcmp(e, "mma") == 0 ? kMma : std::strcmp(e, "tc") == 0 ? kTc : kNone;
}

int64_t workspace_mma(int64_t rows, int group, int head_dim, int requests, bool fp8, cudaError_t &e)
{
    const int wr = attn::row_warps(rows, group, requests);
    switch (head_dim) {
    case 64: return attn::workspace_d<64>(wr, fp8, e);
    case 128: return attn::workspace_d<128>(wr, fp8, e);
    default: return attn::workspace_d<256>(wr, fp8, e);
    }
}

}  // namespace

// enough for every kernel that the launch may choose
int64_t tree_attention_workspace(int64_t rows, int num_heads, int num_kv_heads, int head_dim, int requests, bool fp8,
                                 cudaError_t &e)
{
    const int group = num_heads / num_kv_heads;
    const Pin pin = pinned(head_dim);
    int64_t n = 0;
    if (pin != kTc)
        n = workspace_mma(rows, group, head_dim, requests, fp8, e);
    if (pin == kTc || (pin == kNone && e == cudaSuccess && rows * group > kTcRows * requests)) {
        const int64_t m = head_dim == 64 ? attn::workspace_tc<64>(fp8, e) : attn::workspace_tc<128>(fp8, e);
        n = n > m ? n : m;
    }
    return n;
}

cudaError_t launch_tree_attention(const AttnParams &p, int head_dim, bool fp8, cudaStream_t stream)
{
    const Pin pin = pinned(head_dim);
    bool tc = pin == kTc;
    if (pin == kNone && p.num_rows * p.group > kTcRows * p.num_requests) {
        int dev = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return e;
        const int64_t tiles = (p.table_blocks * p.block_size + 127) / 128;
        tc = tiles * p.num_requests * p.num_kv_heads > sms / 2;
    }
    if (tc)
        return head_dim == 64 ? attn::attention_tc_d<64>(p, fp8, stream) : attn::attention_tc_d<128>(p, fp8, stream);
    const int wr = attn::row_warps(p.num_rows, p.group, p.num_requests);
    switch (head_dim) {
    case 64: return attn::attention_d<64>(p, wr, fp8, stream);
    case 128: return attn::attention_d<128>(p, wr, fp8, stream);
    default: return attn::attention_d<256>(p, wr, fp8, stream);
    }
}

}  // namespace dspark
