// The attention weight the cached tokens received, on the 5th-generation
// tensor cores (tcgen05 + tensor memory, sm_103a).
//
// Mathematics.  For each context token j of a (request, KV head):
//   w_j = decay w_j + sum over the query rows r of e^(scale q_r.k_j - lse_r)
// with the rows of tree_attn_mma.cuh (token r / G, head r % G) and lse as the
// attention left it: the statistics are known, so one pass over K gives it.
//
// Why this shape.  The scores are formed transposed, S = K Q^T with the 128
// keys of a tile as the product's rows: a thread then holds all scores of one
// key in its lane of tensor memory and sums them without any exchange, each
// weight has one owner and one order of summation, and V is not read.  With
// the queries as rows (mma.sync, shuffles and shared memory to sum over rows)
// 64 requests x 7 tokens x 8 heads took 165 us, two long fp8 contexts 184 us.
//
// One CTA per SM takes an equal share of the tiles of all (request, KV head)
// pairs.  Producer warps gather K through the block table into a ring (as in
// tree_attn_tc.cuh), one warp issues the products, two warpgroups of
// 128 threads (one key each) take every other tile from their own buffer of
// scores.  The rows' lse (negated, base 2) and scale sit in shared memory and
// are read as broadcasts.  Heads of more than kRows query rows take them in
// groups, each a pass over the CTA's tiles that adds to what the one before
// wrote (in order: a group's products wait for all sums of the one before).
// Bound: the read of K (64 requests x 7 tokens x 8 heads: 96 us, 70 of it the
// bytes' time); over fp8 the conversion of the tiles (two contexts of 65k to
// 131k tokens: 51 us against 17).
#pragma once

#include "tc_ptx.cuh"
#include "tree_attn_mma.cuh"

namespace dspark {
namespace attn {

constexpr int kWKeys = 128, kWItemCost = 3;

template <int D, bool FP8>
struct WeightTc {
    static constexpr int kRows = D == 256 ? 128 : 256;     // query rows of a group
    static constexpr int kTileBytes = kWKeys * D * 2;
    static constexpr int kStages = D == 256 ? 2 : FP8 ? 384 / D : 512 / D;
    // Warps 0-7 sum, kProducers gather, the last issues.  A bf16 tile is
    // gathered by four, 32 rows each.  An fp8 tile, which waits for its codes
    // and is converted, by two of six that take turns in pairs (four, a tile
    // each, were busy 8,100 cycles with one: 55 us on two long contexts); more
    // than 16 warps would leave the sums 96 registers.
    static constexpr int kProducers = FP8 && D < 256 ? 6 : 4, kGroups = !FP8 ? 1 : D < 256 ? 3 : 2;
    static constexpr int kWarpRows = 128 * kGroups / kProducers;  // rows of a tile per producer warp
    static constexpr int kIssuer = 8 + kProducers, kThreads = 32 * (kIssuer + 1);
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kRow = 2 * D * (FP8 ? 1 : 2);     // bytes of a cached token
    static constexpr int kSmem = 1024 + kQBytes + kStages * kTileBytes;
    static_assert(kSmem + 8 * 1024 <= 227 * 1024 && kStages % kGroups == 0, "shared memory");
};

// This CTA's share: per pair kWItemCost units and a unit per (tile, row group).
template <int ROWS>
struct WeightWalk {
    int64_t lo, hi, at;
    int b, h, tiles, t0, t1, groups;
    Request rq;

    __device__ __forceinline__ static Request checked(const AttnParams &p, int b, unsigned &flags)
    {
        Request r = request(p, b, 0x7fffffff, flags);
        const int q1 = __ldg(p.query_start + b + 1);
        const bool left_out = r.nq == 0 && !(q1 == r.q0 && r.q0 >= 0 && q1 <= p.num_rows);
        if (r.ctx > p.weight_stride || r.ctx > p.table_blocks * p.block_size)
            flags |= kFlagLength, r.ctx = 0;
        if (left_out || r.ctx < 0)
            r.ctx = 0;
        return r;
    }
    __device__ __forceinline__ static int groups_of(const AttnParams &p, const Request &r)
    {
        return max(1, (r.nq * p.group + ROWS - 1) / ROWS);  // a request without drafted tokens decays
    }
    __device__ __forceinline__ static int64_t units(const AttnParams &p, const Request &r)
    {
        if (r.ctx == 0)
            return 0;
        return (int64_t)p.num_kv_heads * ((int64_t)((r.ctx + kWKeys - 1) / kWKeys) * groups_of(p, r) + kWItemCost);
    }
    __device__ __forceinline__ void enter(const AttnParams &p)
    {
        unsigned ignore = 0;
        rq = checked(p, b, ignore);
        tiles = (rq.ctx + kWKeys - 1) / kWKeys;
        groups = groups_of(p, rq);
    }
    __device__ __forceinline__ int64_t span() const { return (int64_t)tiles * groups + kWItemCost; }
    __device__ __forceinline__ void clip()
    {
        const int64_t first = at + kWItemCost, all = (int64_t)tiles * groups;
        t0 = (int)((max((int64_t)0, min(all, lo - first)) + groups - 1) / groups);
        t1 = (int)((max((int64_t)0, min(all, hi - first)) + groups - 1) / groups);
    }
    __device__ __forceinline__ bool more() const { return at < hi; }
    __device__ __forceinline__ void next(const AttnParams &p)
    {
        do {
            at += span();
            if (at >= hi)
                return;
            if (++h >= p.num_kv_heads) {
                h = 0;
                do {
                    b++;
                    enter(p);
                } while (tiles == 0);  // at < hi: there is one
            }
            clip();
        } while (t0 >= t1);
    }
    __device__ __forceinline__ void start(const AttnParams &p, int64_t lo_, int64_t hi_, int first, int64_t before)
    {
        lo = lo_, hi = hi_, at = lo_, b = first;
        h = t0 = t1 = 0;
        if (lo >= hi)
            return;
        enter(p);
        h = (int)Shares::div(lo - before, span());
        at = before + (int64_t)h * span();
        clip();
        if (t0 >= t1)
            next(p);
    }
};

template <int D, bool FP8>
__global__ void __launch_bounds__((WeightTc<D, FP8>::kThreads), 1) weight_kernel(const __grid_constant__ AttnParams p)
{
    using C = WeightTc<D, FP8>;
    using namespace tc;
    constexpr int NS = C::kStages, kRows = C::kRows;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (tc::saddr(smem_raw) & 1023u)) & 1023u);
    unsigned char *sq = smem, *sk = smem + C::kQBytes;
    __shared__ uint64_t kfull[NS], kempty[NS], sfull[2], sempty[2], qfull, qempty, done;
    constexpr int PG = C::kGroups, WR = C::kWarpRows, RG = WR / 32;
    __shared__ uint32_t tmem_slot, live[16][4], rows[C::kProducers][2][WR];
    __shared__ int abort_flag;
    __shared__ int silent[2];  // group number + 1 where a group has rows that saw nothing
    __shared__ __align__(16) float zneg[2][kRows], cscale[2][FP8 ? kRows : 4];  // of a group's rows: -lse, scale (base 2)
    __shared__ int64_t scratch[C::kThreads / 32 + 4];
    const Patience limit{&abort_flag, p.wait_ns};

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < NS; s++) {
            bar_init(kfull + s, C::kProducers / PG * 33);  // a group's copies, and its live masks
            bar_init(kempty + s, 1);
        }
        for (int s = 0; s < 2; s++) {
            bar_init(sfull + s, 1);
            bar_init(sempty + s, 4);
        }
        bar_init(&qfull, 256);
        bar_init(&qempty, 1);
        bar_init(&done, 1);
        abort_flag = silent[0] = silent[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::saddr(&tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_enter();
    unsigned flags = 0;
    using W = WeightWalk<kRows>;
    const int ctas = gridDim.x, cta = blockIdx.x;
    const Find f = find_request<C::kThreads>(p.num_requests, scratch, [&](int b) { return W::units(p, W::checked(p, b, flags)); });
    const Shares shares(f.total, ctas);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;
    W w;
    w.start(p, f.b >= 0 ? shares.start(cta) : 0, f.b >= 0 ? shares.start(cta + 1) : 0, f.b, f.before);

    if (warp == C::kIssuer) {
        // ------------------------------------------------------------ the issuing warp
        const bool leader = elect();
        int x = 0, ng = 0;  // tiles, groups so far
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = ok && bar_wait(bar, parity, limit);
            ok = __all_sync(0xffffffffu, ok);
        };
        while (w.more() && ok) {
            const int n = w.t1 - w.t0, all = w.rq.nq * p.group;
#pragma unroll 1
            for (int row0 = 0; row0 < all && ok; row0 += kRows, ng++) {
                // columns of the product: the group's rows, a multiple of 16
                const uint32_t id = idesc(FP8, false, 128, (min(kRows, all - row0) + 15) & ~15);
                wait(&qfull, (uint32_t)ng & 1u);
#pragma unroll 1
                for (int j = 0; j < n && ok; j++, x++) {
                    const int st = x % NS, buf = x & 1;
                    wait(kfull + st, (uint32_t)(x / NS) & 1u);
                    wait(sempty + buf, ((uint32_t)(x >> 1) & 1u) ^ 1u);
                    if (!ok)
                        break;
                    fence_async();
                    fence_after();
                    if (leader) {
                        pick<NS>(st, [&](auto stc) {
                            pick<2>(buf, [&](auto bc) {
                                constexpr int S = decltype(stc)::value, B = decltype(bc)::value;
                                const uint32_t a = tc::saddr(sk) + S * C::kTileBytes, b = tc::saddr(sq);
#pragma unroll
                                for (int k = 0; k < D / 16; k++)
                                    mma_ss(tmem + 256 * B, desc128(a + (k / 4) * 16384 + (k % 4) * 32, 16),
                                           desc128(b + (k / 4) * (kRows * 128) + (k % 4) * 32, 16), id, k != 0);
                                mma_commit(sfull + B);
                                mma_commit(kempty + S);
                            });
                        });
                    }
                    __syncwarp();
                }
                if (leader)
                    mma_commit(&qempty);
                __syncwarp();
            }
            w.next(p);
        }
        if (leader)
            mma_commit(&done);
        __syncwarp();
    } else if (warp >= 8) {
        // ------------------------------------------------------------ producers (a tile is gathered once per row group)
        const int pw = warp - 8, mine = pw % PG, row0 = pw / PG * WR;  // tiles number mine, mine + PG, ...; rows row0 ...
        struct Cursor {
            W w;
            int tile, group;
            __device__ __forceinline__ void skip(const AttnParams &p)  // pairs without query rows have no products
            {
                while (w.more() && w.rq.nq == 0)
                    w.next(p);
                tile = w.t0, group = 0;
            }
            __device__ __forceinline__ void step(const AttnParams &p)
            {
                if (++tile >= w.t1) {
                    tile = w.t0;
                    if (++group >= w.groups) {
                        w.next(p);
                        skip(p);
                    }
                }
            }
        };
        Cursor lk;
        lk.w = w;
        lk.skip(p);
        for (int i = 0; i < mine && lk.w.more(); i++)
            lk.step(p);
        int phys[RG], off[RG], look_h = 0, looked = 0;  // looked: tiles looked up, two ahead while there are any
        auto look = [&]() {
#pragma unroll
            for (int g = 0; g < RG; g++)
                off[g] = -1;
            if (!lk.w.more())
                return;
            looked++;
            look_h = lk.w.h;
#pragma unroll
            for (int g = 0; g < RG; g++) {
                const int j = lk.tile * kWKeys + row0 + 32 * g + lane, blk = block_of(p, j);
                phys[g] = 0;
                if (j < lk.w.rq.ctx) {
                    off[g] = j - blk * p.block_size;
                    phys[g] = __ldg(p.table + lk.w.b * p.table_stride + blk);
                }
            }
            for (int i = 0; i < PG && lk.w.more(); i++)
                lk.step(p);
        };
        auto resolve = [&](int slot) {
#pragma unroll
            for (int g = 0; g < RG; g++) {
                uint32_t at = ~0u;
                if (off[g] >= 0) {
                    if (phys[g] < 0 || phys[g] >= p.num_blocks) {
                        flags |= kFlagBlockRange;
                    } else {
                        at = (uint32_t)(((int64_t)phys[g] * p.num_kv_heads + look_h) * p.block_size + off[g]);
                        const unsigned char *row = p.cache + (int64_t)at * C::kRow;
#pragma unroll
                        for (int y = 0; y < C::kRow / 2; y += 128)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(row + y));
                    }
                }
                rows[pw][slot][32 * g + lane] = at;
            }
            __syncwarp();
        };
        constexpr int kW = D * (FP8 ? 1 : 2) / 16;  // 16-byte words of a row's K
        constexpr int kIt = WR * kW / 32, kB = kIt < 8 ? kIt : 8;  // words per lane, so many at a time
        bool ok = true;
        look();
        resolve(0);
        look();
        if (p.test_hold)
            looked = 0;  // test hook: nothing is copied, the other roles' waits run out
        for (int i = 0; i < looked && ok; i++) {
            const int x = mine + PG * i, st = x % NS;
            const uint32_t dst0 = tc::saddr(sk) + st * C::kTileBytes;
            const uint32_t *from = rows[pw][i & 1];
            resolve((i & 1) ^ 1);
            look();
            ok = bar_wait(kempty + st, ((uint32_t)(x / NS) & 1u) ^ 1u, limit);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
#pragma unroll 1
            for (int i0 = 0; i0 < kIt; i0 += kB) {
                uint32_t src[kB];
#pragma unroll
                for (int k = 0; k < kB; k++)
                    src[k] = from[((i0 + k) * 32 + lane) / kW];
#pragma unroll
                for (int k = 0; k < kB; k++) {
                    const int y = row0 + ((i0 + k) * 32 + lane) / kW, c = ((i0 + k) * 32 + lane) % kW;
                    const uint32_t at = FP8 ? raw_at<D>(dst0, y, c) : dst0 + (c >> 3) * 16384 + y * 128 + (((c & 7) ^ (y & 7)) << 4);
                    cp16(at, src[k] != ~0u ? p.cache + (int64_t)src[k] * C::kRow + 16 * c : p.cache, src[k] != ~0u);
                }
            }
#pragma unroll
            for (int g = 0; g < RG; g++) {
                const unsigned bits = __ballot_sync(0xffffffffu, from[32 * g + lane] != ~0u);
                if (lane == 0)
                    live[x & 15][row0 / 32 + g] = bits;
            }
            if constexpr (FP8) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                convert_rows<D, WR>(dst0, row0, kWKeys);
                fence_async();
            }
            if (lane == 0)
                bar_arrive(kfull + st);  // the live mask
            if (FP8)
                bar_arrive(kfull + st);
            else
                bar_arrive_copies(kfull + st);
            __syncwarp();  // every lane is done with this tile's row numbers
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ------------------------------------------------------------ the sums: a thread per key
        const int e = warp >> 2, q4 = warp & 3, r = q4 * 32 + lane;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const float ks = FP8 && p.k_scale ? __ldg(p.k_scale) : 1.0f;
        const float base_scale = p.scale * kLog2e * ks;
        const uint64_t c2 = pr(base_scale, base_scale);
        int x = 0, ng = 0;
        bool ok = true;
        while (w.more() && ok) {
            const int n = w.t1 - w.t0, all = w.rq.nq * p.group;
            float *weights = p.weights + ((int64_t)w.b * p.num_kv_heads + w.h) * p.weight_stride;
            if (all == 0) {  // nothing but the decay; a tile per warpgroup
                for (int j = e; j < n; j += 2) {
                    const int key = (w.t0 + j) * kWKeys + r;
                    if (key < w.rq.ctx)
                        weights[key] *= p.decay;
                }
            }
            for (int row0 = 0; row0 < all && ok; row0 += kRows, ng++) {
                const int cols = min(kRows, all - row0), zb = ng & 1;
                // ---- the group's rows: thread tid takes row row0 + tid, once no product reads the last ones
                if (ng > 0) {
                    ok = bar_wait(&qempty, (uint32_t)(ng - 1) & 1u, limit);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok)
                        break;
                }
                if (tid < kRows) {
                    const int row = row0 + tid;
                    const bool mine = row < all;
                    const int i = mine ? row / p.group : 0, hq = w.h * p.group + (mine ? row - i * p.group : 0);
                    const uint16_t *src = p.q + (int64_t)(w.rq.q0 + i) * p.q_ts + (int64_t)hq * p.q_hs;
                    float inv = 1.0f, fix = 1.0f;
                    // a row that saw nothing, or none at all, adds nothing whatever its scores hold
                    const float lse = mine ? __ldg(p.lse + (int64_t)(w.rq.q0 + i) * p.num_heads + hq) : -INFINITY;
                    zneg[zb][tid] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
                    if (mine && lse == -INFINITY)
                        silent[zb] = ng + 1;
                    if constexpr (FP8) {
                        float top = 0.0f;
                        if (mine)
#pragma unroll 8
                            for (int k = 0; k < D / 8; k++) {
                                const uint4 q = __ldg(reinterpret_cast<const uint4 *>(src) + k);
                                const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                                for (int m = 0; m < 4; m++)
                                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qw[m] << 16)), fabsf(__uint_as_float(qw[m] & 0xffff0000u))));
                            }
                        int ex = 0;
                        if (top > 0.0f && top < __int_as_float(0x7f800000))
                            ex = max(ilogbf(top), -126);
                        cscale[zb][tid] = base_scale * scalbnf(1.0f, ex);
                        inv = scalbnf(1.0f, ex > 126 ? -126 : -ex);
                        fix = ex > 126 ? 0.5f : 1.0f;
                    }
                    const uint32_t dst0 = tc::saddr(sq);
#pragma unroll 8
                    for (int k = 0; k < D / 8; k++) {
                        uint4 q = make_uint4(0, 0, 0, 0);
                        if (mine)
                            q = __ldg(reinterpret_cast<const uint4 *>(src) + k);
                        uint32_t qw[4] = {q.x, q.y, q.z, q.w};
                        if constexpr (FP8) {
#pragma unroll
                            for (int m = 0; m < 4; m++)
                                qw[m] = pack2<true>(__uint_as_float(qw[m] << 16) * inv * fix, __uint_as_float(qw[m] & 0xffff0000u) * inv * fix);
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst0 + (k >> 3) * (kRows * 128) + tid * 128 + (((k & 7) ^ (tid & 7)) << 4)),
                                     "r"(qw[0]), "r"(qw[1]), "r"(qw[2]), "r"(qw[3])
                                     : "memory");
                    }
                    fence_async();
                }
                bar_arrive(&qfull);
                // ---- every other tile of this share
#pragma unroll 1
                for (int j = 0; j < n; j++, x++) {
                    if ((x & 1) != e)
                        continue;
                    const int key = (w.t0 + j) * kWKeys + r;
                    const bool first = row0 == 0;
                    float old = 0.0f;
                    if (first && key < w.rq.ctx)
                        old = weights[key];
                    ok = bar_wait(sfull + e, (uint32_t)(x >> 1) & 1u, limit);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok)
                        break;
                    fence_after();
                    // what the group before wrote, maybe in the other warpgroup:
                    // this group's scores came after all of that
                    if (!first && key < w.rq.ctx)
                        old = weights[key];
                    uint64_t s0 = 0, s1 = 0;
                    const bool mute = silent[zb] == ng + 1;
#pragma unroll 1
                    for (int c0 = 0; c0 < cols; c0 += 32) {
                        uint32_t y[32];
                        tmem_ld32(tmem + lanes + 256 * e + c0, y);
                        const float4 *z = reinterpret_cast<const float4 *>(zneg[zb] + c0);
                        const float4 *cs = reinterpret_cast<const float4 *>(cscale[zb] + (FP8 ? c0 : 0));
                        const bool some = cols - c0 < 32 || mute;  // some of the columns count for nothing
#pragma unroll
                        for (int k = 0; k < 8; k++) {
                            const float4 zv = z[k];
                            uint64_t f0 = c2, f1 = c2;
                            if constexpr (FP8) {
                                const float4 cv = cs[k];
                                f0 = pr(cv.x, cv.y), f1 = pr(cv.z, cv.w);
                            }
                            float a0, a1, a2, a3;
                            unpr(fma2(pr(__uint_as_float(y[4 * k]), __uint_as_float(y[4 * k + 1])), f0, pr(zv.x, zv.y)), a0, a1);
                            unpr(fma2(pr(__uint_as_float(y[4 * k + 2]), __uint_as_float(y[4 * k + 3])), f1, pr(zv.z, zv.w)), a2, a3);
                            a0 = ex2(a0), a1 = ex2(a1), a2 = ex2(a2), a3 = ex2(a3);
                            if (some) {
                                a0 = zv.x != -INFINITY ? a0 : 0.0f, a1 = zv.y != -INFINITY ? a1 : 0.0f;
                                a2 = zv.z != -INFINITY ? a2 : 0.0f, a3 = zv.w != -INFINITY ? a3 : 0.0f;
                            }
                            s0 = add2(s0, pr(a0, a1));
                            s1 = add2(s1, pr(a2, a3));
                        }
                    }
                    fence_before();
                    const bool here = (live[x & 15][q4] >> lane) & 1u;
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(sempty + e);  // the scores (and the tile's live bits) are read
                    if (key < w.rq.ctx) {
                        float a, b2;
                        unpr(add2(s0, s1), a, b2);
                        const float sum = here ? a + b2 : 0.0f;  // nothing for a token in a block out of range
                        weights[key] = first ? fmaf(p.decay, old, sum) : old + sum;
                    }
                }
            }
            w.next(p);
        }
    }
    __syncthreads();
    if (warp == C::kIssuer) {
        if (lane == 0) {
            const unsigned long long t0 = gtimer();
            while (!bar_try(&done, 0) && !(flags & kFlagTimeout))
                if (gtimer() - t0 > limit.ns)
                    flags |= kFlagTimeout;
        }
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
    if (tid == 0 && *limit.abort)
        flags |= kFlagTimeout;
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0 && flags && p.error_flags)
        atomicOr(p.error_flags, flags);
}

template <int D, bool FP8>
cudaError_t weight(const AttnParams &p, cudaStream_t stream)
{
    using C = WeightTc<D, FP8>;
    static int cached[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    int have = __atomic_load_n(&cached[dev], __ATOMIC_ACQUIRE);
    if (have == 0) {
        e = cudaDeviceGetAttribute(&have, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(weight_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess)
            return e;
        __atomic_store_n(&cached[dev], have, __ATOMIC_RELEASE);
    }
    return launch_pdl(weight_kernel<D, FP8>, have, C::kThreads, C::kSmem, stream, p);
}

}  // namespace attn
}  // namespace dspark
