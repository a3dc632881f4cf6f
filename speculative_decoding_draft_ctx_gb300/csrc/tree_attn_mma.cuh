// Drafted tokens' attention over the paged cache: the pieces that its kernels
// and the weight accumulation share, and the attention kernel for up to 64
// query rows at a time (mma.sync, sm_103a).
//
// Mathematics.  For a query row q and the keys j it sees, with s_j = scale
// q.k_j:  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),  lse = m +
// log sum_j e^(s_j - m), for any m.  Keys are taken tile by tile with m the
// maximum so far (less a constant, next paragraph); when it grows, the sums
// are multiplied by e^(m_old - m).  Two results over disjoint keys join the
// same way, so the keys of one query row can be split over warps and CTAs.
// Exponentials are base 2 with log2(e) folded into the scale.  Scores,
// statistics and sums are fp32.
//
// Rounding of the weights.  For the second product the weights 2^(s - m) are
// rounded to the type of the tile: bf16 over a bf16 cache, each by at most
// 2^-8 of itself against weights summed unrounded; fp16 over an fp8 cache,
// whose codes are exact in fp16, by at most 2^-11 of itself while it is a
// normal number.  fp16 has normal numbers from 2^-14 on and 15 octaves above
// 1, so m is the maximum less kLift = 14 there: the largest weight is 2^14, a
// weight keeps its 2^-11 down to 2^-28 of the largest (below, it is off by at
// most 2^-39 of the largest).  With the largest at 1 a thin tail behind one
// heavy token lost its bits below 2^-14 and vanished below 2^-25, while the
// sum still counted it (32,768 tokens with 0.03% of the weight: all of it).
//
// Rows and items.  The G query heads of a KV head and the drafted tokens of a
// request are the rows of one matrix: row r is token r / G, head r % G, so K|V
// are read once for all of them.  An item is R = 16 WR such rows of one
// (request, KV head); its unit is one tile of 64 keys.  Lengths are on the
// device, so each CTA sums the units over the requests itself and takes an
// equal share of the flattened unit sequence, whatever the lengths are: a
// long request is split over many CTAs, many short ones share one.  An item
// that lies in one CTA's share is finished there; of a split one every CTA
// writes its part (unnormalised sum, m and sum of weights, fp32) and a second
// kernel, launched with programmatic overlap, joins the parts in the order of
// the CTAs.  There are no atomics: the same inputs give the same bits.
//
// Tiles.  K|V of a token are one contiguous row of the cache, gathered with
// 16-byte asynchronous copies (one row per warp instruction at 512 bytes)
// through the block table, whose entries are fetched one tile ahead; any
// block size works, a page may end inside a tile.  Rows past the end and rows
// in blocks out of range arrive as zeros and are masked.  16-byte words of
// row x sit at word ^ swz(x) so that every shared-memory read below is free
// of bank conflicts.  Four warps: WR of them along rows, WK = 4 / WR along
// the keys of a tile (few rows leave the tensor cores idle anyway; splitting
// the keys lets all four warps convert and exponentiate), joined through
// shared memory when the item ends.
//
// fp8.  Codes become fp16 exactly.  K: a lane reads 16 neighbouring bytes of
// a key, which serve as its operands of four products of depth 16; that
// permutes the depth index, so q is loaded in the same order.  V: ldmatrix
// transposes byte pairs, so one 8 x 16 byte matrix gives the operands of the
// even and of the odd dims.  q is scaled per row by a power of two to below
// 2 before its (then exact, but for what lies 2^-24 below the row's largest)
// conversion to fp16, and the scores by its inverse.
//
// What a row does not see.  Scores of masked keys are replaced by -inf
// whatever they are; V rows of drafted tokens that hold infinities or NaN are
// zeroed in the tile, and the results of the rows that do see them are set
// to what such a value makes of a sum.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "ctx_kv_device.cuh"
#include "ctx_kv_internal.h"
#include "draft_attn_internal.h"

namespace dspark {
namespace attn {

constexpr int kThreads = 128, kWarps = 4, kTile = 64;
constexpr int kItemCost = 4;  // of an item besides its tiles, in tiles of kTile keys (see Walk)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLift = 14.0f;             // of the weights over an fp8 cache, in octaves
constexpr float kLiftBelow = 1048576.0f;   // scores from here on are too coarse to take kLift off

// The m that a row with this maximum (base 2) subtracts.  From 2^20 on steps
// of fp32 are an eighth and more: m - kLift could round to beyond fp16's
// range, so such a maximum is taken as it is.
template <bool FP8>
__device__ __forceinline__ float reference_of(float top)
{
    return FP8 && fabsf(top) < kLiftBelow ? top - kLift : top;
}

__device__ __forceinline__ uint32_t saddr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16-byte words of row x are stored at word ^ swz(x): eight consecutive rows
// use eight different words (ldmatrix), rows 2i and 2i + 1 differ in bit 2
// (four neighbouring words of both rows at once: the fp8 key reads).
__device__ __forceinline__ int swz(int x)
{
    return ((x & 1) << 2) | ((x >> 1) & 3);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live)
{
    const int n = live ? 16 : 0;  // the rest of the 16 bytes is filled with zeros
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// two e4m3 codes (low 16 bits of w) -> an fp16 pair, exactly
__device__ __forceinline__ uint32_t e4m3_to_half2(uint16_t w)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        return pack_bf16x2(lo, hi);
    }
}

// ------------------------------------------------------------------ requests, items, units

// j / block_size by a multiply (p.block_magic = floor(2^64 / block_size) + 1, exact while j * block_size < 2^64; 0 for size 1)
__device__ __forceinline__ int block_of(const AttnParams &p, int j)
{
    return p.block_magic ? (int)__umul64hi((unsigned long long)j, p.block_magic) : j;
}

struct Request {
    int q0, nq, ctx;  // first row of q, drafted tokens, context tokens (nq = 0: nothing to do)
};

// Request b, checked; flags collects what is wrong.
__device__ __forceinline__ Request request(const AttnParams &p, int b, int mask_limit, unsigned &flags)
{
    const int q0 = __ldg(p.query_start + b), q1 = __ldg(p.query_start + b + 1), ctx = __ldg(p.context_lens + b);
    Request r{q0, q1 - q0, ctx};
    const bool bad = q0 < 0 || q1 < q0 || q1 > p.num_rows || ctx < 0 ||
                     (q1 > q0 && ((int64_t)ctx + (q1 - q0) > p.table_blocks * p.block_size || q1 - q0 > mask_limit));
    if (bad) {
        flags |= kFlagLength;
        r.nq = 0;
    }
    return r;
}

// n CTAs share `total` units: CTA c gets [start(c), start(c + 1)), the first
// `more` of them one unit more.
struct Shares {
    int64_t each;
    int more, n;

    __device__ __forceinline__ static int64_t div(int64_t a, int64_t b)  // of nonnegative numbers; most fit 32 bits
    {
        return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
    }
    __device__ __forceinline__ Shares(int64_t total, int ctas)
    {
        n = total < ctas ? (int)total : ctas;
        each = n ? div(total, n) : 0;
        more = (int)(total - each * n);
    }
    __device__ __forceinline__ int64_t start(int c) const { return c < n ? each * c + min(c, more) : each * n + more; }
    __device__ __forceinline__ int owner(int64_t unit) const  // the CTA whose share holds it
    {
        const int64_t edge = (each + 1) * more;
        return (int)(unit < edge ? div(unit, each + 1) : more + div(unit - edge, each));
    }
};

// Block-wide search (THREADS threads, scratch of THREADS / 32 + 4 words) of the
// request that holds this CTA's first unit: `units(b)` is evaluated by one thread.
struct Find {
    int64_t total, before;  // all units; those of the requests before `b`
    int b;                  // < 0: the CTA has no share
};

template <int THREADS, typename F>
__device__ __forceinline__ Find find_request(int requests, int64_t *scratch, F units)
{
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Find f{0, 0, -1};
    int64_t base = 0, mine = 0, end = 0;  // before this chunk of THREADS requests; of this thread's; up to and with it
    auto scan = [&](int b0) {
        const int b = b0 + tid;
        mine = b < requests ? units(b) : 0;
        int64_t x = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d)
                x += y;
        }
        if (b0)
            __syncthreads();
        if (lane == 31)
            scratch[warp] = x;
        __syncthreads();
        // each warp sums the warps' totals with its own lanes
        int64_t t = lane < W ? scratch[lane] : 0, all = t;
        t = lane < warp ? t : 0;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
            t += __shfl_xor_sync(0xffffffffu, t, d);
            all += __shfl_xor_sync(0xffffffffu, all, d);
        }
        end = base + t + x;
        base += all;
    };
    for (int b0 = 0; b0 < requests; b0 += THREADS)
        scan(b0);
    f.total = base;
    const int64_t target = Shares(base, gridDim.x).start(blockIdx.x);
    if ((int64_t)blockIdx.x >= base)  // fewer units than CTAs
        return f;
    auto hit = [&](int b0) {
        if (target >= end - mine && target < end) {
            scratch[W] = b0 + tid;
            scratch[W + 1] = end - mine;
        }
    };
    if (requests <= THREADS) {
        hit(0);
    } else {
        base = 0;
        __syncthreads();
        for (int b0 = 0; b0 < requests; b0 += THREADS) {
            scan(b0);
            hit(b0);
        }
    }
    __syncthreads();
    f.b = (int)scratch[W];
    f.before = scratch[W + 1];
    return f;
}

// The flattened sequence of work: for every request, for every item (a row
// group of ROWS of one KV head), EXTRA units for what an item costs besides its
// tiles (queries in, results out, an empty pipeline: without them a CTA that
// got two dozen requests of a few tokens took as long as all others together),
// then a unit per tile.  A CTA's share [lo, hi) of it gives it the tiles of an
// item whose units lie inside.
template <int ROWS, int KEYS, int EXTRA>
struct Walk {
    int64_t lo, hi, at;  // the share; where the current item begins
    int b, item, items, tiles, t0, t1, groups;  // t0 .. t1: this CTA's tiles of the item
    int mask_limit;
    Request rq;

    __device__ __forceinline__ static int64_t units(const AttnParams &p, const Request &r)
    {
        if (r.nq == 0)
            return 0;
        const int64_t items = (int64_t)p.num_kv_heads * (((int64_t)r.nq * p.group + ROWS - 1) / ROWS);
        return items * ((r.ctx + r.nq + KEYS - 1) / KEYS + EXTRA);
    }
    __device__ __forceinline__ void enter(const AttnParams &p)
    {
        unsigned ignore = 0;
        rq = request(p, b, mask_limit, ignore);
        groups = (rq.nq * p.group + ROWS - 1) / ROWS;
        items = rq.nq ? p.num_kv_heads * groups : 0;
        tiles = (rq.ctx + rq.nq + KEYS - 1) / KEYS;
    }
    __device__ __forceinline__ void clip()
    {
        const int64_t first = at + EXTRA;
        t0 = (int)max((int64_t)0, min((int64_t)tiles, lo - first));
        t1 = (int)max((int64_t)0, min((int64_t)tiles, hi - first));
    }
    __device__ __forceinline__ bool more() const { return at < hi; }
    // to the next item with tiles of this CTA; at >= hi when there is none
    __device__ __forceinline__ void next(const AttnParams &p)
    {
        do {
            at += tiles + EXTRA;
            if (at >= hi)
                return;
            if (++item >= items) {
                item = 0;
                do {
                    b++;
                    enter(p);
                } while (items == 0);  // at < hi: there is one
            }
            clip();
        } while (t0 >= t1);
    }
    // the first item of the share of request `first`, whose units begin at `before`
    __device__ __forceinline__ void start(const AttnParams &p, int64_t lo_, int64_t hi_, int first, int64_t before, int limit)
    {
        lo = lo_, hi = hi_, at = lo_, b = first, mask_limit = limit;
        item = t0 = t1 = 0;
        if (lo >= hi)
            return;
        enter(p);
        item = (int)Shares::div(lo - before, tiles + EXTRA);
        at = before + (int64_t)item * (tiles + EXTRA);
        clip();
        if (t0 >= t1)
            next(p);
    }
    __device__ __forceinline__ int head() const { return item / groups; }
    __device__ __forceinline__ int row0() const { return (item % groups) * ROWS; }
    __device__ __forceinline__ bool begun() const { return t0 == 0; }
    __device__ __forceinline__ bool finished() const { return t1 == tiles; }
    // the CTA that has the item's last tile
    __device__ __forceinline__ int last_cta(const Shares &shares) const { return shares.owner(at + EXTRA + tiles - 1); }
};

// ------------------------------------------------------------------ the cached tiles

// Copies kTile rows of `ROW` bytes of one (request, KV head) into a stage,
// through the block table.  A warp takes 16
// rows; its lanes 0..15 (and 16..31 alike) hold the block of their row, which
// `fetch` has read for the tile that `load` will copy next.
template <int ROW>
struct Loader {
    static constexpr int kWords = ROW / 16;
    int64_t phys;
    int off;
    bool live;

    __device__ __forceinline__ void fetch(const AttnParams &p, int b, int tile, int len)
    {
        const int j = tile * kTile + (threadIdx.x >> 5) * 16 + (threadIdx.x & 15);
        live = j < len;
        phys = 0;
        off = 0;
        if (live) {
            const int blk = block_of(p, j);
            off = j - blk * p.block_size;
            phys = __ldg(p.table + b * p.table_stride + blk);
        }
    }

    // live bits of the warp's 16 rows go to mask[warp]
    __device__ __forceinline__ void load(const AttnParams &p, int h, uint32_t stage, uint32_t *mask, unsigned &flags)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (live && (phys < 0 || phys >= p.num_blocks)) {
            flags |= kFlagBlockRange;
            live = false;
        }
        const unsigned bits = __ballot_sync(0xffffffffu, live) & 0xffffu;
        if (lane == 0)
            mask[warp] = bits;
        const unsigned char *row =
            p.cache + (live ? ((phys * p.num_kv_heads + h) * p.block_size + off) * (int64_t)ROW : 0);
        constexpr int kIt = 16 * kWords / 32, kBatch = kIt < 8 ? kIt : 8;
#pragma unroll
        for (int i0 = 0; i0 < kIt; i0 += kBatch) {  // the addresses, then the copies: the shuffles' latency once
            unsigned long long src[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; i++)
                src[i] = __shfl_sync(0xffffffffu, (unsigned long long)row, ((i0 + i) * 32 + lane) / kWords);
#pragma unroll
            for (int i = 0; i < kBatch; i++) {
                const int idx = (i0 + i) * 32 + lane;
                const int x = idx / kWords, c = idx % kWords, y = warp * 16 + x;
                cp16(stage + y * ROW + ((c ^ swz(y)) << 4), reinterpret_cast<const unsigned char *>(src[i]) + 16 * c,
                     (bits >> x) & 1u);
            }
        }
    }
};

// whether a 32-bit word of V holds an infinity or NaN
__device__ __forceinline__ bool nonfinite_word(uint32_t w, bool fp8)
{
    if (fp8) {  // any byte 0x7f or 0xff
        const uint32_t x = (w & 0x7f7f7f7fu) ^ 0x7f7f7f7fu;
        return ((x - 0x01010101u) & ~x & 0x80808080u) != 0;
    }
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// ------------------------------------------------------------------ fp8 tiles of the tensor-core kernels

// A tile's operand holds a row of D fp16 values as D / 64 pieces of 128 bytes,
// 16384 bytes apart, 16-byte words of row y at word ^ (y & 7).  The row's D
// codes are copied into the upper half of the row's own bytes (word c at
// raw_at) and converted from there in place: no row touches another's bytes,
// and a short rolled loop does it (from registers, unrolled, a 16-byte word
// took 330 cycles of a warp, mostly instruction fetches).
template <int D>
__device__ __forceinline__ uint32_t raw_at(uint32_t tile, int y, int c)
{
    return tile + (D == 64 ? 0 : (D / 128 + (c >> 3)) * 16384) + y * 128 + ((c & 7) << 4);
}

// Rows [row0, row0 + ROWS) of a tile by one warp, after their codes have
// landed.  Rows from `clean` on have NaN codes zeroed; true if there were any.
template <int D, int ROWS>
__device__ __forceinline__ bool convert_rows(uint32_t tile, int row0, int clean)
{
    constexpr int kW = D / 16, kR = 32 / kW, kU = kR < 8 ? 8 / kR : 1, kStep = kU * kR;  // whole groups of 8 rows a step
    const int lane = threadIdx.x & 31, c = lane % kW, r = lane / kW;
    bool any = false;
    if (clean < row0 + ROWS) {
#pragma unroll 1
        for (int y = row0 + r; y < row0 + ROWS; y += kR)
#pragma unroll 1
            for (int k = 0; k < 4 && y >= clean; k++) {
                const uint32_t at = raw_at<D>(tile, y, c) + 4 * k;
                uint32_t q;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(q) : "r"(at) : "memory");
                if (nonfinite_word(q, true)) {
                    any = true;
#pragma unroll 1
                    for (int e = 0; e < 32; e += 8)
                        if (((q >> e) & 0x7fu) == 0x7fu)
                            q &= ~(0xffu << e);
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(q) : "memory");
                }
            }
        __syncwarp();
    }
    // 16-byte words 2 c and 2 c + 1 of the fp16 row, odd lanes the other way
    // round (bank conflicts)
    uint32_t from[kU], to[kU][2];
#pragma unroll
    for (int u = 0; u < kU; u++) {
        const int y = row0 + u * kR + r;
        from[u] = raw_at<D>(tile, y, c);
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const int cc = 2 * c + (k ^ (c & 1));
            to[u][k] = tile + (cc >> 3) * 16384 + y * 128 + (((cc & 7) ^ (y & 7)) << 4);
        }
    }
#pragma unroll 1
    for (int d = 0; d < ROWS * 128; d += kStep * 128) {
        uint32_t q[kU][4];
#pragma unroll
        for (int u = 0; u < kU; u++)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(q[u][0]), "=r"(q[u][1]), "=r"(q[u][2]), "=r"(q[u][3])
                         : "r"(from[u] + d)
                         : "memory");
        __syncwarp();  // the rows' codes are read before their bytes are written
#pragma unroll
        for (int u = 0; u < kU; u++)
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const bool upper = (k != 0) != ((c & 1) != 0);
                const uint32_t a = upper ? q[u][2] : q[u][0], b = upper ? q[u][3] : q[u][1];
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to[u][k] + d), "r"(e4m3_to_half2((uint16_t)a)),
                             "r"(e4m3_to_half2((uint16_t)(a >> 16))), "r"(e4m3_to_half2((uint16_t)b)),
                             "r"(e4m3_to_half2((uint16_t)(b >> 16)))
                             : "memory");
            }
    }
    return any;
}

// ------------------------------------------------------------------ queries

// The A operands of a warp's 16 rows: reg 0 / 1 row g / g + 8 of the lower 8
// depths, reg 2 / 3 of the upper 8.  bf16: the plain depth order.  fp8: the
// order of the key reads, and `row_scale` (2 rows) the power of two that was
// taken out.
template <int D, bool FP8>
__device__ __forceinline__ void load_q(const AttnParams &p, const Request &rq, int h, int row0, uint32_t (&a)[D / 16][4],
                                       float (&row_scale)[2])
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rows = rq.nq * p.group;
#pragma unroll
    for (int s = 0; s < 2; s++) {
        const int r = row0 + g + 8 * s;
        row_scale[s] = 1.0f;
        const bool live = r < rows;
        const int i = live ? r / p.group : 0;
        const uint16_t *src = p.q + (int64_t)(rq.q0 + i) * p.q_ts + (int64_t)(h * p.group + (live ? r - i * p.group : 0)) * p.q_hs;
        if constexpr (!FP8) {
#pragma unroll
            for (int k = 0; k < D / 16; k++) {
                a[k][s] = live ? *reinterpret_cast<const uint32_t *>(src + 16 * k + 2 * t) : 0u;
                a[k][2 + s] = live ? *reinterpret_cast<const uint32_t *>(src + 16 * k + 8 + 2 * t) : 0u;
            }
        } else {
            uint32_t w[D / 8];
            float top = 0.0f;
#pragma unroll
            for (int u = 0; u < D / 64; u++) {
#pragma unroll
                for (int v = 0; v < 2; v++) {
                    const uint4 x = live ? *reinterpret_cast<const uint4 *>(src + 64 * u + 16 * t + 8 * v) : make_uint4(0, 0, 0, 0);
                    w[8 * u + 4 * v] = x.x, w[8 * u + 4 * v + 1] = x.y, w[8 * u + 4 * v + 2] = x.z, w[8 * u + 4 * v + 3] = x.w;
                }
            }
#pragma unroll
            for (int u = 0; u < D / 8; u++)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[u] << 16)), fabsf(__uint_as_float(w[u] & 0xffff0000u))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            int e = 0;
            if (top > 0.0f && top < __int_as_float(0x7f800000))
                e = ilogbf(top);
            row_scale[s] = scalbnf(1.0f, e < -126 ? -126 : e);
            const float inv = scalbnf(1.0f, e > 126 ? -126 : -(e < -126 ? -126 : e));
            const float fix = e > 126 ? 0.5f : 1.0f;  // 2^-127 as 2^-126 / 2
#pragma unroll
            for (int u = 0; u < D / 64; u++)
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uint32_t x = w[8 * u + 2 * k], y = w[8 * u + 2 * k + 1];
                    a[4 * u + k][s] = pack2<true>(__uint_as_float(x << 16) * inv * fix, __uint_as_float(x & 0xffff0000u) * inv * fix);
                    a[4 * u + k][2 + s] = pack2<true>(__uint_as_float(y << 16) * inv * fix, __uint_as_float(y & 0xffff0000u) * inv * fix);
                }
        }
    }
}

// s[i] += 16 query rows x the 8 keys from key0 + 8 i, PITCH bytes per stage row, K at its start
template <int D, bool FP8, int NT, int PITCH>
__device__ __forceinline__ void scores(float (&s)[NT][4], const uint32_t (&a)[D / 16][4], uint32_t stage, int key0)
{
    const int lane = threadIdx.x & 31;
    if constexpr (!FP8) {
        // ldmatrix x4: keys 0-7 / 8-15 of a pair of n-tiles, depth words c and c + 1
        const int key = key0 + (lane & 7) + ((lane >> 4) << 3), w = (lane >> 3) & 1;
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
            const int x = key + 8 * i;
            const uint32_t row = stage + x * PITCH;
            const int z = swz(x);
#pragma unroll
            for (int k = 0; k < D / 16; k++) {
                uint32_t b[4];
                ldsm4(b, row + (((2 * k + w) ^ z) << 4));
                mma<false>(s[i], a[k], b[0], b[1]);
                mma<false>(s[i + 1], a[k], b[2], b[3]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NT; i++) {
            const int x = key0 + 8 * i + (lane >> 2);
            const uint32_t row = stage + x * PITCH;
            const int z = swz(x);
#pragma unroll
            for (int u = 0; u < D / 64; u++) {
                uint32_t w[4];
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(row + (((4 * u + (lane & 3)) ^ z) << 4))
                             : "memory");
#pragma unroll
                for (int k = 0; k < 4; k++)
                    mma<true>(s[i], a[4 * u + k], e4m3_to_half2((uint16_t)w[k]), e4m3_to_half2((uint16_t)(w[k] >> 16)));
            }
        }
    }
}

// ------------------------------------------------------------------ the attention kernel

template <int D, bool FP8, int WR>
struct Cfg {
    static constexpr int kWK = kWarps / WR, kRows = 16 * WR, kKeys = kTile / kWK;  // keys of a tile per warp
    static constexpr int kRow = 2 * D * (FP8 ? 1 : 2);                            // bytes of a token's K|V
    static constexpr int kStage = kTile * kRow;
    // CTAs per SM by registers (about 250 a thread at D 128 and 256, 168 at 64),
    // and as many stages as share the SM's shared memory between them
    static constexpr int kCtas = D == 64 ? 3 : D == 128 ? 2 : 1;
    static constexpr int kStages = D == 64 ? (FP8 ? 6 : 4) : D == 128 ? (FP8 ? 5 : 2) : (FP8 ? 4 : 2);
    static constexpr int kNT = D / 8;                                            // n-tiles of the output
    static constexpr int kJoin = kWK > 1 ? (kWK / 2) * WR * (kNT * 128 + 64) * 4 : 0;  // bytes to join the key warps
    static constexpr int kSmem = kStages * kStage + kJoin;
    static constexpr int kPart = WR * (kNT * 128 + 32);                          // floats of one part
    static_assert(kCtas * (kSmem + 1536) <= 227 * 1024, "shared memory");
};

// What a CTA tells the join about the item it began and did not finish.
struct PartDesc {
    int32_t q0, rows, row0, h;  // the request's first q row, its rows (nq G), the item's first, KV head
    int32_t last;               // the last CTA with a part of it; < 0: there is no such item
    int32_t nq, ctx, b;
    int32_t bad[2];             // this CTA's parts 0 and 1: did infinities or NaN among the drafted V come up
    int32_t pad[2];
};

// What p.parts holds: ctas descriptors, then 2 parts per CTA (0: of an item
// begun before it, 1: of the item it begins and does not finish).  A part is
// per row warp: kNT x 4 x 32 accumulators as the lanes hold them, then 16 m
// and 16 sums.

__device__ __forceinline__ bool sees(const AttnParams &p, const Request &rq, int i, int a)
{
    if (a < 0)
        return true;  // context
    if (a >= rq.nq)
        return false;
    if (p.mask_kind == 0)
        return true;
    if (p.mask_kind == 1)
        return a <= i;
    return (__ldg(p.tree_mask + (int64_t)(rq.q0 + i) * p.mask_words + (a >> 6)) >> (a & 63)) & 1ull;
}

// V[a, d] of the request's drafted token a as a float (0 where its block is out of range)
template <int D, bool FP8>
__device__ __forceinline__ float drafted_v(const AttnParams &p, int b, int ctx, int h, int a, int d)
{
    const int j = ctx + a, blk = j / p.block_size;
    const int64_t phys = __ldg(p.table + b * p.table_stride + blk);
    if (phys < 0 || phys >= p.num_blocks)
        return 0.0f;
    const int64_t at = ((phys * p.num_kv_heads + h) * p.block_size + (j - blk * p.block_size)) * (2 * D) + D + d;
    if (FP8) {
        const uint32_t c = e4m3_to_half2(p.cache[at]);
        return __half2float(__ushort_as_half((unsigned short)(c & 0xffffu)));
    }
    return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p.cache)[at] << 16);
}

// Adds to dims [d0, d1) of row i's result `dst` what the infinities and NaN
// among the drafted V it sees make of the sum (their tile entries were zeroed).
template <int D, bool FP8>
__device__ __noinline__ void add_nonfinite(const AttnParams &p, int b, Request rq, int h, int i, uint16_t *dst, int d0, int d1)
{
    for (int d = d0; d < d1; d++) {
        float x = 0.0f;
        for (int a = 0; a < rq.nq; a++) {
            if (!sees(p, rq, i, a))
                continue;
            const float v = drafted_v<D, FP8>(p, b, rq.ctx, h, a, d);
            if (!(fabsf(v) <= 3.4028235e38f))
                x += v;
        }
        if (x != 0.0f)  // NaN too
            dst[d] = (uint16_t)pack_bf16x2(__uint_as_float((uint32_t)dst[d] << 16) + x, 0.0f);
    }
}

template <int D, bool FP8, int WR>
__global__ void __launch_bounds__(kThreads, (Cfg<D, FP8, WR>::kCtas)) attention_kernel(const __grid_constant__ AttnParams p)
{
    using C = Cfg<D, FP8, WR>;
    constexpr int NS = C::kKeys / 8;  // n-tiles of a warp's scores
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t scratch[kWarps + 4];
    __shared__ uint32_t live[C::kStages][kWarps];
    __shared__ int any_bad;
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wr = warp % WR, wk = warp / WR;
    const int g = lane >> 2;
    const uint32_t stages = saddr(smem);
    float *join = reinterpret_cast<float *>(smem + C::kStages * C::kStage);
    unsigned flags = 0;
    const int mask_limit = p.mask_kind == 2 ? 64 * p.mask_words : 0x7fffffff;

    // ---- this CTA's share of the units
    const int ctas = gridDim.x, cta = blockIdx.x;
    using W = Walk<C::kRows, kTile, kItemCost>;
    const Find f = find_request<kThreads>(p.num_requests, scratch,
                                          [&](int b) { return W::units(p, request(p, b, mask_limit, flags)); });
    const Shares shares(f.total, ctas);
    PartDesc *descs = reinterpret_cast<PartDesc *>(p.parts);
    float *parts = p.parts + (int64_t)ctas * (sizeof(PartDesc) / 4);
    if (tid == 0)
        descs[cta].last = -1, descs[cta].bad[0] = 0, descs[cta].bad[1] = 0;
    if (f.b < 0) {
        flags = __reduce_or_sync(0xffffffffu, flags);
        if (flags && lane == 0 && p.error_flags)
            atomicOr(p.error_flags, flags);
        return;
    }
    const float ks = FP8 && p.k_scale ? __ldg(p.k_scale) : 1.0f, vs = FP8 && p.v_scale ? __ldg(p.v_scale) : 1.0f;
    const float base_scale = p.scale * kLog2e * ks;

    // ---- two walks over the share: one for the copies, one for the products
    W w;
    w.start(p, shares.start(cta), shares.start(cta + 1), f.b, f.before, mask_limit);
    W cp = w;
    int cp_tile = cp.t0;

    Loader<C::kRow> ld;
    if (cp.more())
        ld.fetch(p, cp.b, cp_tile, cp.rq.ctx + cp.rq.nq);
    auto issue = [&](int stage) {
        if (cp.more()) {
            ld.load(p, cp.head(), stages + stage * C::kStage, live[stage], flags);
            if (++cp_tile >= cp.t1) {
                cp.next(p);
                cp_tile = cp.t0;
            }
            if (cp.more())
                ld.fetch(p, cp.b, cp_tile, cp.rq.ctx + cp.rq.nq);
        }
        cp_commit();
    };
#pragma unroll
    for (int s = 0; s < C::kStages - 1; s++)
        issue(s);
    int stage = 0;

    while (w.more()) {
        // ---------------------------------------------------------------- one item, as far as it is this CTA's
        const int h = w.head(), row0 = w.row0();
        const int len = w.rq.ctx + w.rq.nq, rows = w.rq.nq * p.group;
        const Request rq = w.rq;
        const int b = w.b;
        uint32_t qa[D / 16][4];
        float rs[2];
        load_q<D, FP8>(p, rq, h, row0 + 16 * wr, qa, rs);
        const float c0 = base_scale * rs[0], c1 = base_scale * rs[1];
        const int r0 = row0 + 16 * wr + g, i0 = r0 / p.group, i1 = (r0 + 8) / p.group;
        float o[C::kNT][4];
#pragma unroll
        for (int n = 0; n < C::kNT; n++)
            o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        if (tid == 0)
            any_bad = 0;

        for (int tile = w.t0; tile < w.t1; tile++) {
            cp_wait<C::kStages - 2>();
            __syncthreads();  // the tile has landed for all; every warp is done with the stage that is filled next
            issue((stage + C::kStages - 1) % C::kStages);
            const uint32_t st = stages + stage * C::kStage;
            const int key0 = tile * kTile;
            const bool drafted = key0 + kTile > rq.ctx;  // the tile holds drafted tokens or ends beyond them
            if (drafted) {
                // infinities and NaN among the drafted V: zeroed here, accounted for at the end
                for (int x = tid; x < kTile * (C::kRow / 32); x += kThreads) {
                    const int y = x / (C::kRow / 32), c = C::kRow / 32 + x % (C::kRow / 32);
                    if (key0 + y < rq.ctx || key0 + y >= len)
                        continue;
                    uint4 *at = reinterpret_cast<uint4 *>(smem + stage * C::kStage + y * C::kRow + ((c ^ swz(y)) << 4));
                    uint4 v = *at;
                    uint32_t vw[4] = {v.x, v.y, v.z, v.w};
                    bool hit = false;
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if (nonfinite_word(vw[k], FP8)) {
                            hit = true;
                            if (FP8) {
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    if (((vw[k] >> (8 * e)) & 0x7fu) == 0x7fu)
                                        vw[k] &= ~(0xffu << (8 * e));
                            } else {
                                if ((vw[k] & 0x7f80u) == 0x7f80u)
                                    vw[k] &= 0xffff0000u;
                                if ((vw[k] & 0x7f800000u) == 0x7f800000u)
                                    vw[k] &= 0xffffu;
                            }
                        }
                    if (hit) {
                        *at = make_uint4(vw[0], vw[1], vw[2], vw[3]);
                        any_bad = 1;
                    }
                }
                __syncthreads();
            }
            float s[NS][4];
#pragma unroll
            for (int n = 0; n < NS; n++)
                s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
            scores<D, FP8, NS, C::kRow>(s, qa, st, wk * C::kKeys);
            const uint32_t lv[4] = {live[stage][0], live[stage][1], live[stage][2], live[stage][3]};
            const bool masked = drafted || (lv[0] & lv[1] & lv[2] & lv[3]) != 0xffffu;
#pragma unroll
            for (int n = 0; n < NS; n++) {
                s[n][0] = __fmul_rn(s[n][0], c0), s[n][1] = __fmul_rn(s[n][1], c0);  // rounded apart from the
                s[n][2] = __fmul_rn(s[n][2], c1), s[n][3] = __fmul_rn(s[n][3], c1);  // subtraction of m: exactly 0 at the maximum
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int y = wk * C::kKeys + 8 * n + 2 * (lane & 3) + e;
                        const int a = key0 + y - rq.ctx;
                        const bool in = (lv[y >> 4] >> (y & 15)) & 1u;
                        if (!in || !(r0 < rows && sees(p, rq, i0, a)))
                            s[n][e] = -INFINITY;
                        if (!in || !(r0 + 8 < rows && sees(p, rq, i1, a)))
                            s[n][2 + e] = -INFINITY;
                    }
                }
            }
            // ---- softmax statistics
            float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
            for (int n = 0; n < NS; n++) {
                t0 = fmaxf(t0, fmaxf(s[n][0], s[n][1]));
                t1 = fmaxf(t1, fmaxf(s[n][2], s[n][3]));
            }
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
            t0 = fmaxf(m0, reference_of<FP8>(t0)), t1 = fmaxf(m1, reference_of<FP8>(t1));
            const float u0 = t0 == -INFINITY ? 0.0f : t0, u1 = t1 == -INFINITY ? 0.0f : t1;  // nothing seen yet
            const float f0 = ex2(m0 - u0), f1 = ex2(m1 - u1);
            m0 = t0, m1 = t1;
            float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
            for (int n = 0; n < NS; n++) {
                s[n][0] = ex2(s[n][0] - u0), s[n][1] = ex2(s[n][1] - u0);
                s[n][2] = ex2(s[n][2] - u1), s[n][3] = ex2(s[n][3] - u1);
                a0 += s[n][0] + s[n][1];
                a1 += s[n][2] + s[n][3];
            }
            l0 = fmaf(l0, f0, a0), l1 = fmaf(l1, f1, a1);  // this lane's columns; joined over the quad at the end
            if (__any_sync(0xffffffffu, f0 != 1.0f || f1 != 1.0f)) {
#pragma unroll
                for (int n = 0; n < C::kNT; n++)
                    o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
            }
            // ---- o += p V
#pragma unroll
            for (int j = 0; j < NS / 2; j++) {
                const uint32_t pa[4] = {pack2<FP8>(s[2 * j][0], s[2 * j][1]), pack2<FP8>(s[2 * j][2], s[2 * j][3]),
                                        pack2<FP8>(s[2 * j + 1][0], s[2 * j + 1][1]),
                                        pack2<FP8>(s[2 * j + 1][2], s[2 * j + 1][3])};
                const int x = wk * C::kKeys + 16 * j + (lane & 15);
                const uint32_t row = st + x * C::kRow;
                const int z = swz(x);
                if constexpr (!FP8) {
#pragma unroll
                    for (int n = 0; n < D / 16; n++) {  // 16 dims: words 2 n and 2 n + 1 of V
                        uint32_t v[4];
                        ldsm4t(v, row + (((D / 8 + 2 * n + (lane >> 4)) ^ z) << 4));
                        mma<false>(o[2 * n], pa, v[0], v[1]);
                        mma<false>(o[2 * n + 1], pa, v[2], v[3]);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < D / 32; n++) {  // 32 dims: words 2 n and 2 n + 1 of V, 16 dims each
                        uint32_t v[4];
                        ldsm4t(v, row + (((D / 16 + 2 * n + (lane >> 4)) ^ z) << 4));
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            // bytes (dim 2n, dim 2n+1) of key 2t, then of key 2t + 1
                            const uint32_t x0 = __byte_perm(v[2 * k], 0, 0x3120), x1 = __byte_perm(v[2 * k + 1], 0, 0x3120);
                            mma<true>(o[4 * n + 2 * k], pa, e4m3_to_half2((uint16_t)x0), e4m3_to_half2((uint16_t)x1));
                            mma<true>(o[4 * n + 2 * k + 1], pa, e4m3_to_half2((uint16_t)(x0 >> 16)), e4m3_to_half2((uint16_t)(x1 >> 16)));
                        }
                    }
                }
            }
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
        }

        // ---------------------------------------------------------------- the item ends here, or the CTA's share does
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1), l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2), l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if constexpr (C::kWK > 1) {
            // pairs of key warps, the upper half into the lower
#pragma unroll
            for (int half = C::kWK / 2; half >= 1; half /= 2) {
                __syncthreads();
                float *at = join + ((wk % half) * WR + wr) * (C::kNT * 128 + 64);
                if (wk >= half && wk < 2 * half) {
#pragma unroll
                    for (int n = 0; n < C::kNT; n++)
#pragma unroll
                        for (int c = 0; c < 4; c++)
                            at[(n * 4 + c) * 32 + lane] = o[n][c];
                    if ((lane & 3) == 0) {
                        at[C::kNT * 128 + g] = m0, at[C::kNT * 128 + 8 + g] = m1;
                        at[C::kNT * 128 + 16 + g] = l0, at[C::kNT * 128 + 24 + g] = l1;
                    }
                }
                __syncthreads();
                if (wk < half) {
                    const float om0 = at[C::kNT * 128 + g], om1 = at[C::kNT * 128 + 8 + g];
                    const float ol0 = at[C::kNT * 128 + 16 + g], ol1 = at[C::kNT * 128 + 24 + g];
                    const float t0 = fmaxf(m0, om0), t1 = fmaxf(m1, om1);
                    const float u0 = t0 == -INFINITY ? 0.0f : t0, u1 = t1 == -INFINITY ? 0.0f : t1;
                    const float x0 = ex2(m0 - u0), x1 = ex2(m1 - u1), y0 = ex2(om0 - u0), y1 = ex2(om1 - u1);
                    l0 = l0 * x0 + ol0 * y0, l1 = l1 * x1 + ol1 * y1;
                    m0 = t0, m1 = t1;
#pragma unroll
                    for (int n = 0; n < C::kNT; n++) {
                        o[n][0] = o[n][0] * x0 + at[(n * 4 + 0) * 32 + lane] * y0;
                        o[n][1] = o[n][1] * x0 + at[(n * 4 + 1) * 32 + lane] * y0;
                        o[n][2] = o[n][2] * x1 + at[(n * 4 + 2) * 32 + lane] * y1;
                        o[n][3] = o[n][3] * x1 + at[(n * 4 + 3) * 32 + lane] * y1;
                    }
                }
            }
        }
        const bool begun = w.begun(), done = w.finished();
        const int bad = any_bad;
        if (wk == 0) {
            if (begun && done) {
                const float inv0 = l0 > 0.0f ? vs / l0 : l0 == 0.0f ? 0.0f : l0, inv1 = l1 > 0.0f ? vs / l1 : l1 == 0.0f ? 0.0f : l1;
#pragma unroll
                for (int sx = 0; sx < 2; sx++) {
                    const int r = r0 + 8 * sx;
                    if (r >= rows)
                        continue;
                    const int i = sx ? i1 : i0, hq = h * p.group + (r - i * p.group);
                    uint16_t *dst = p.out + ((int64_t)(rq.q0 + i) * p.num_heads + hq) * D;
                    const float inv = sx ? inv1 : inv0;
                    if ((lane & 3) == 0) {
                        const float l = sx ? l1 : l0, m = sx ? m1 : m0;
                        p.lse[(int64_t)(rq.q0 + i) * p.num_heads + hq] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
                    }
#pragma unroll
                    for (int n = 0; n < C::kNT; n += 2) {
                        const float x[4] = {o[n][2 * sx] * inv, o[n][2 * sx + 1] * inv, o[n + 1][2 * sx] * inv, o[n + 1][2 * sx + 1] * inv};
                        if constexpr (FP8) {
                            // dims 16 (n / 2) + 4 t ...: even tile, odd tile, even, odd
                            *reinterpret_cast<uint2 *>(dst + 8 * n + 4 * (lane & 3)) = make_uint2(pack_bf16x2(x[0], x[2]), pack_bf16x2(x[1], x[3]));
                        } else {
                            *reinterpret_cast<uint32_t *>(dst + 8 * n + 2 * (lane & 3)) = pack_bf16x2(x[0], x[1]);
                            *reinterpret_cast<uint32_t *>(dst + 8 * n + 8 + 2 * (lane & 3)) = pack_bf16x2(x[2], x[3]);
                        }
                    }
                }
                if (bad) {
                    __syncwarp();  // the rows are written: one lane of each four adds to them
                    if ((lane & 3) == 0) {
                        if (r0 < rows)
                            add_nonfinite<D, FP8>(p, b, rq, h, i0, p.out + ((int64_t)(rq.q0 + i0) * p.num_heads + h * p.group + (r0 - i0 * p.group)) * D, 0, D);
                        if (r0 + 8 < rows)
                            add_nonfinite<D, FP8>(p, b, rq, h, i1, p.out + ((int64_t)(rq.q0 + i1) * p.num_heads + h * p.group + (r0 + 8 - i1 * p.group)) * D, 0, D);
                    }
                    __syncwarp();
                }
            } else {
                float *part = parts + ((int64_t)cta * 2 + (begun ? 1 : 0)) * C::kPart + wr * (C::kNT * 128 + 32);
#pragma unroll
                for (int n = 0; n < C::kNT; n++)
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        part[(n * 4 + c) * 32 + lane] = o[n][c];
                if ((lane & 3) == 0) {
                    part[C::kNT * 128 + g] = m0, part[C::kNT * 128 + 8 + g] = m1;
                    part[C::kNT * 128 + 16 + g] = l0, part[C::kNT * 128 + 24 + g] = l1;
                }
            }
        }
        if (begun && !done && tid == 0) {
            PartDesc &d = descs[cta];
            d.q0 = rq.q0, d.rows = rows, d.row0 = row0, d.h = h, d.nq = rq.nq, d.ctx = rq.ctx, d.b = b;
            d.last = w.last_cta(shares);
        }
        if (bad && !(begun && done) && tid == 0)
            descs[cta].bad[begun ? 1 : 0] = 1;
        __syncthreads();  // any_bad and the join buffer are free again
        w.next(p);
    }
    cp_wait<0>();
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && lane == 0 && p.error_flags)
        atomicOr(p.error_flags, flags);
}

// Joins the parts of the item that CTA blockIdx.x of the attention kernel
// began and did not finish; block y joins row warp y, its four warps a
// quarter of the dims each.
template <int D, bool FP8, int WR>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ AttnParams p, int ctas)
{
    using C = Cfg<D, FP8, WR>;
    constexpr int NW = C::kNT / kWarps;  // n-tiles per warp (an even number)
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, wr = blockIdx.y;
    const PartDesc *descs = reinterpret_cast<const PartDesc *>(p.parts);
    const PartDesc d = descs[blockIdx.x];
    const int row0 = d.row0 + 16 * wr;
    if (d.last < 0 || row0 >= d.rows)
        return;
    const float *parts = p.parts + (int64_t)ctas * (sizeof(PartDesc) / 4);
    constexpr int kWarpPart = C::kNT * 128 + 32;
    auto part = [&](int c) {
        return parts + ((int64_t)c * 2 + (c == (int)blockIdx.x ? 1 : 0)) * C::kPart + wr * kWarpPart;
    };
    // loads of several parts at a time: one after the other, an item over 19
    // CTAs took 30 us to join
    const int first = blockIdx.x;
    float t0 = -INFINITY, t1 = -INFINITY;
    bool bad = false;
    for (int c0 = first; c0 <= d.last; c0 += 8) {
        float v0[8], v1[8];
        int any[8];
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int c = min(c0 + k, d.last);
            v0[k] = part(c)[C::kNT * 128 + g], v1[k] = part(c)[C::kNT * 128 + 8 + g];
            any[k] = descs[c].bad[c == first ? 1 : 0];
        }
#pragma unroll
        for (int k = 0; k < 8; k++)
            t0 = fmaxf(t0, v0[k]), t1 = fmaxf(t1, v1[k]), bad |= any[k] != 0;
    }
    const float u0 = t0 == -INFINITY ? 0.0f : t0, u1 = t1 == -INFINITY ? 0.0f : t1;
    float l0 = 0.0f, l1 = 0.0f, o[NW][4];
#pragma unroll
    for (int n = 0; n < NW; n++)
        o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    for (int c0 = first; c0 <= d.last; c0 += 4) {
        float v[4][NW][4], ml[4][4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const bool there = c0 + k <= d.last;
            const float *at = part(there ? c0 + k : d.last);
#pragma unroll
            for (int x = 0; x < 4; x++)
                ml[k][x] = there ? at[C::kNT * 128 + 8 * x + g] : x < 2 ? -INFINITY : 0.0f;
#pragma unroll
            for (int n = 0; n < NW; n++)
#pragma unroll
                for (int x = 0; x < 4; x++)
                    v[k][n][x] = there ? at[(warp * NW + n) * 128 + 32 * x + lane] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float x0 = ex2(ml[k][0] - u0), x1 = ex2(ml[k][1] - u1);
            l0 = fmaf(ml[k][2], x0, l0), l1 = fmaf(ml[k][3], x1, l1);
#pragma unroll
            for (int n = 0; n < NW; n++) {
                o[n][0] = fmaf(v[k][n][0], x0, o[n][0]), o[n][1] = fmaf(v[k][n][1], x0, o[n][1]);
                o[n][2] = fmaf(v[k][n][2], x1, o[n][2]), o[n][3] = fmaf(v[k][n][3], x1, o[n][3]);
            }
        }
    }
    const float vs = FP8 && p.v_scale ? __ldg(p.v_scale) : 1.0f;
#pragma unroll
    for (int s = 0; s < 2; s++) {
        const int r = row0 + g + 8 * s;
        if (r >= d.rows)
            continue;
        const int i = r / p.group, hq = d.h * p.group + (r - i * p.group);
        const float l = s ? l1 : l0, m = s ? t1 : t0;
        const float inv = l > 0.0f ? vs / l : l == 0.0f ? 0.0f : l;
        const int64_t at = (int64_t)(d.q0 + i) * p.num_heads + hq;
        if (warp == 0 && (lane & 3) == 0)
            p.lse[at] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
        uint16_t *dst = p.out + at * D;
#pragma unroll
        for (int k = 0; k < NW; k += 2) {
            const int n = warp * NW + k;
            const float x[4] = {o[k][2 * s] * inv, o[k][2 * s + 1] * inv, o[k + 1][2 * s] * inv, o[k + 1][2 * s + 1] * inv};
            if constexpr (FP8) {
                *reinterpret_cast<uint2 *>(dst + 8 * n + 4 * (lane & 3)) = make_uint2(pack_bf16x2(x[0], x[2]), pack_bf16x2(x[1], x[3]));
            } else {
                *reinterpret_cast<uint32_t *>(dst + 8 * n + 2 * (lane & 3)) = pack_bf16x2(x[0], x[1]);
                *reinterpret_cast<uint32_t *>(dst + 8 * n + 8 + 2 * (lane & 3)) = pack_bf16x2(x[2], x[3]);
            }
        }
    }
    if (bad) {
        __syncwarp();  // the warp's quarter of each row is written: one lane of each four adds to it
        if ((lane & 3) == 0)
            for (int s = 0; s < 2; s++) {
                const int r = row0 + g + 8 * s, i = r / p.group;
                if (r < d.rows)
                    add_nonfinite<D, FP8>(p, d.b, Request{d.q0, d.nq, d.ctx}, d.h, i,
                                          p.out + ((int64_t)(d.q0 + i) * p.num_heads + d.h * p.group + (r - i * p.group)) * D,
                                          warp * (D / 4), (warp + 1) * (D / 4));
            }
    }
}

// ------------------------------------------------------------------ launches

template <typename K>
cudaError_t prepare(K kernel, int smem, int per_sm_most, int &ctas)
{
    int dev = 0, sms = 0, per = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, smem);
    ctas = sms * (per < 1 ? 1 : per > per_sm_most ? per_sm_most : per);
    return e;
}

// The attention's CTAs for this variant on the current device (cached).
template <int D, bool FP8, int WR>
cudaError_t attention_ctas(int &ctas)
{
    static int cached[64];  // written with the same value by whoever comes first
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    int have = __atomic_load_n(&cached[dev], __ATOMIC_ACQUIRE);
    if (have == 0) {
        using C = Cfg<D, FP8, WR>;
        e = prepare(attention_kernel<D, FP8, WR>, C::kSmem, C::kCtas, have);
        if (e != cudaSuccess)
            return e;
        __atomic_store_n(&cached[dev], have, __ATOMIC_RELEASE);
    }
    ctas = have;
    return cudaSuccess;
}

template <int D, bool FP8, int WR>
int64_t attention_bytes(cudaError_t &e)
{
    int ctas = 0;
    e = attention_ctas<D, FP8, WR>(ctas);
    return e == cudaSuccess ? (int64_t)ctas * ((int64_t)sizeof(PartDesc) + 2 * (int64_t)Cfg<D, FP8, WR>::kPart * 4) : 0;
}

template <int D, bool FP8, int WR>
cudaError_t attention(const AttnParams &p, cudaStream_t stream)
{
    using C = Cfg<D, FP8, WR>;
    int ctas = 0;
    cudaError_t e = attention_ctas<D, FP8, WR>(ctas);
    if (e != cudaSuccess)
        return e;
    e = launch_pdl(attention_kernel<D, FP8, WR>, ctas, kThreads, C::kSmem, stream, p);
    if (e != cudaSuccess)
        return e;
    return launch_pdl_grid(join_kernel<D, FP8, WR>, dim3((unsigned)ctas, (unsigned)WR), kThreads, 0, 0, stream, p, ctas);
}

// Rows of an item: the smallest of 16, 32 and 64 that holds the mean request's
// rows, 64 beyond.  Lengths are on the device; rows / requests is what the
// host knows of them.
inline int row_warps(int64_t rows, int group, int requests)
{
    const int64_t mean = (rows * group + requests - 1) / requests;
    return mean <= 16 ? 1 : mean <= 32 ? 2 : 4;
}

template <int D>
int64_t workspace_d(int wr, bool fp8, cudaError_t &e)
{
    switch (wr) {
    case 1: return fp8 ? attention_bytes<D, true, 1>(e) : attention_bytes<D, false, 1>(e);
    case 2: return fp8 ? attention_bytes<D, true, 2>(e) : attention_bytes<D, false, 2>(e);
    default: return fp8 ? attention_bytes<D, true, 4>(e) : attention_bytes<D, false, 4>(e);
    }
}

template <int D>
cudaError_t attention_d(const AttnParams &p, int wr, bool fp8, cudaStream_t stream)
{
    switch (wr) {
    case 1: return fp8 ? attention<D, true, 1>(p, stream) : attention<D, false, 1>(p, stream);
    case 2: return fp8 ? attention<D, true, 2>(p, stream) : attention<D, false, 2>(p, stream);
    default: return fp8 ? attention<D, true, 4>(p, stream) : attention<D, false, 4>(p, stream);
    }
}

// one translation unit per head dim
#define DSPARK_ATTN_DECLARE(D)                                                     \
    extern template int64_t workspace_d<D>(int, bool, cudaError_t &);              \
    extern template cudaError_t attention_d<D>(const AttnParams &, int, bool, cudaStream_t);
#define DSPARK_ATTN_DEFINE(D)                                                      \
    template int64_t workspace_d<D>(int, bool, cudaError_t &);                     \
    template cudaError_t attention_d<D>(const AttnParams &, int, bool, cudaStream_t);

}  // namespace attn
}  // namespace dspark
