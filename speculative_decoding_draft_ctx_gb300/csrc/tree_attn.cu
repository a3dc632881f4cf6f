// Which kernel serves a call of the drafted tokens' attention.
#include <cstdlib>
#include <cstring>

#include "tree_attn_tc.cuh"

namespace dspark {
namespace attn {
DSPARK_ATTN_DECLARE(64)
DSPARK_ATTN_DECLARE(128)
DSPARK_ATTN_DECLARE(256)
DSPARK_ATTN_SCALED_DECLARE(64)
DSPARK_ATTN_SCALED_DECLARE(128)
DSPARK_ATTN_SCALED_DECLARE(256)
DSPARK_ATTN_TC_SCALED_DECLARE(64)
DSPARK_ATTN_TC_SCALED_DECLARE(128)
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

// Page-scaled caches: an item of mma.sync has up to 64 rows, and beyond these reads
// the cache again, while the tensor-core kernel is bound by its producers, whose
// time does not depend on the rows.  Measured, mma.sync / tensor cores, us:
//   rows 56, 64 requests x 8 heads over 4,000   D 128 263 / 323, D 64 186 / 274
//   rows 72, the same                           D 128 495 / 327, D 64 349 / 269
//   rows 56, 1 x 8 over 2,000                   D 128 19.9 / 21.6, D 64 18.6 / 19.8
//   rows 72, the same                           D 128 23.5 / 21.9, D 64 19.7 / 19.9
//   rows 504, 1 x 4 over 16,000                 D 128 76 / 45, D 64 56 / 38
constexpr int64_t kTcRowsScaled = 64;

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

// Whether a call of more than `rows` rows a KV head takes the tensor cores.
cudaError_t takes_tc(const AttnParams &p, int head_dim, int64_t rows, bool &tc)
{
    const Pin pin = pinned(head_dim);
    tc = pin == kTc;
    if (pin == kNone && p.num_rows * p.group > rows * p.num_requests) {
        int dev = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return e;
        const int64_t tiles = (p.table_blocks * p.block_size + 127) / 128;
        tc = tiles * p.num_requests * p.num_kv_heads > sms / 2;
    }
    return cudaSuccess;
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
    bool tc = false;
    const cudaError_t e = takes_tc(p, head_dim, kTcRows, tc);
    if (e != cudaSuccess)
        return e;
    if (tc)
        return head_dim == 64 ? attn::attention_tc_d<64>(p, fp8, stream) : attn::attention_tc_d<128>(p, fp8, stream);
    const int wr = attn::row_warps(p.num_rows, p.group, p.num_requests);
    switch (head_dim) {
    case 64: return attn::attention_d<64>(p, wr, fp8, stream);
    case 128: return attn::attention_d<128>(p, wr, fp8, stream);
    default: return attn::attention_d<256>(p, wr, fp8, stream);
    }
}

int64_t tree_attention_scaled_workspace(int64_t rows, int num_heads, int num_kv_heads, int head_dim, int requests, cudaError_t &e)
{
    const int group = num_heads / num_kv_heads, wr = attn::row_warps(rows, group, requests);
    const Pin pin = pinned(head_dim);
    int64_t n = 0;
    if (pin != kTc)
        n = head_dim == 64 ? attn::workspace_scaled_d<64>(wr, e) : head_dim == 128 ? attn::workspace_scaled_d<128>(wr, e)
                                                                             : attn::workspace_scaled_d<256>(wr, e);
    if (pin == kTc || (pin == kNone && e == cudaSuccess && rows * group > kTcRowsScaled * requests)) {
        const int64_t m = head_dim == 64 ? attn::workspace_tc<64>(true, e) : attn::workspace_tc<128>(true, e);
        n = n > m ? n : m;
    }
    return n;
}

cudaError_t launch_tree_attention_scaled(const AttnParams &p, int head_dim, cudaStream_t stream)
{
    bool tc = false;
    const cudaError_t e = takes_tc(p, head_dim, kTcRowsScaled, tc);
    if (e != cudaSuccess)
        return e;
    if (tc)
        return head_dim == 64 ? attn::attention_tc_scaled_d<64>(p, stream) : attn::attention_tc_scaled_d<128>(p, stream);
    const int wr = attn::row_warps(p.num_rows, p.group, p.num_requests);
    switch (head_dim) {
    case 64: return attn::attention_scaled_d<64>(p, wr, stream);
    case 128: return attn::attention_scaled_d<128>(p, wr, stream);
    default: return attn::attention_scaled_d<256>(p, wr, stream);
    }
}

}  // namespace dspark
