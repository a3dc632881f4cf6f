// Attention over page-scaled caches for up to 64 query rows at a time: keys split over
// the warps for the scores, dims for the output (mma.sync, sm_103a).
//
// Mathematics.  A page and head has one power of two for K and one for V, 2^ek and
// 2^ev.  The products take the codes, exact in fp16, as in tree_attn_mma.cuh; a score
// is multiplied by its key's 2^ek, and the weight that the second product takes is
// 2^(s + ev - m), with m of the running maximum of s + ev: rounded as there, relative
// to the largest contribution.  The sum of weights takes 2^-ev of it back, exactly but
// for fp32's own rounding (|ev| <= 32).  A key's scales are read beside its page's
// number one tile before they are stored, so that no load is waited for.
//
// Split.  Items, shares, tiles and the join are those of tree_attn_mma.cuh.  There each
// warp has 16 rows and all dims of its own, so all four of a 64-row item turn all of a
// tile's codes into fp16, and at D 256 the sums of few rows already are 128 registers
// of a thread.  Here a warp takes 16 of a tile's 64 keys for all rows, and a quarter of
// the dims of V over all keys: every code is converted once.  The queries lie in
// shared memory as the lanes take them; so do the weights, written by the warp that has
// their keys as the operands of one product of depth 16, and read by all.
//
// A tile has two barriers.  Behind the first its codes, and the weights of the
// tile before, are there: its scores are taken, the warps' row maxima written,
// and the products with V of the tile before follow, before the second.  Behind that
// all know the common maximum; sums are rescaled, the weights written and the next
// copies issued into the stage that those products have left.
//
// What it measured: 64 requests of 1,024 to 8,192 tokens, 64 query and 8 KV heads, with
// 8 / 32 / 56 rows a KV head, us, and with a warp per 16 rows:
//   D 64    83 / 107 / 168     92 / 122 / 181
//   D 128  107 / 151 / 235    132 / 182 / 272
//   D 256  193 / 367 / 543    335 / 482 / 787
// What bounds it: at 56 rows of D 128 some 830 instructions a warp and tile, a third of
// a warp's time in fixed latencies (products, conversions, shuffles), the barriers
// behind them; shared memory 62%, issue 47%, the tensor pipe 44%.  Few rows are bound by
// the path through a tile, not by bytes: at 8 rows a scheduler's 3.8 warps issue 55% of
// the time, an instruction takes a warp 7 cycles (1.7 fixed latencies, 0.9 barriers, 0.9
// shared memory, 0.7 loads), DRAM is at 36% (D 64) and 56% (D 128).  In a copy with clocks
// read between its steps (D 64 and D 128 alike) the copies had landed but for 50 of some
// 3,000 cycles a tile; issuing the next ones, 16 bytes of a key each, took 1,150, the scores 700.
// With the walk over the requests in every thread's registers the sums of D 256 spilled
// (802 where 583 was taken).
#pragma once

#include "tree_attn_mma.cuh"

namespace dspark {
namespace attn {

// A row's m stays until its maximum has grown by more than an octave, that is, is more
// than kLimit above m (a difference, which is exact for scores of any size): weights
// are up to 2^15 then, fp16 goes to 2^16, and in most tiles no sum is rescaled
// (267 -> 255 us at 56 rows of D 128).  kNothing: m where nothing has been seen, the
// lowest number (no infinity, so that -inf - m is one; no score lies below it, and one
// that equals it weighs 1).
constexpr float kLimit = kLift + 1.0f, kNothing = -3.402823466e38f;

// Units per CTA at least, where that leaves a CTA per SM: every CTA of a long request
// leaves a part to join.  One request of 16,000 tokens, 4 KV heads, us: 8 / 56 rows of D 64
// 57 / 46 with a unit each, 26 / 33 with 4, 24 / 30 with 8; 56 rows of D 128 46, 36, 35;
// but 4 requests of 3,000, 8 KV heads, 56 rows of D 128 take 30, 30 and 33, of D 64 23, 23, 26.
constexpr int kGrain = 4;

template <int D, int RT>  // RT: groups of 16 rows
struct SplitCfg {
    static constexpr int kRows = 16 * RT, kRow = 2 * D, kStage = kTile * kRow;
    static constexpr int kWords = D / 16 / kWarps;  // 16-byte words of V (16 dims each) per warp
    // CTAs per SM by registers and shared memory, stages by what these leave: more warps
    // cover a tile's latencies, more stages gain nothing.  64 requests, us: 8 rows of D 128
    // 107 with 4 CTAs of 3 stages, 117 with 3 of 4, 150 with 2 of 6; of D 64 83 with 4 of
    // 5 or 6, 95 with 3 of 6, 126 with 2 of 10; 32 rows of D 64 107 with 4 of 5, 117 with 3 of
    // 6 or 7, 149 with 2 of 10.
    static constexpr int kCtas = D == 64 ? (RT <= 2 ? 4 : 3) : D == 128 ? (RT == 1 ? 4 : 3) : RT == 1 ? 2 : 1;
    static constexpr int kStages = D == 64 ? (RT == 2 ? 5 : 6) : D == 128 ? 3 : RT == 1 ? 3 : 5;
    static constexpr int kPlans = 8;  // items planned at once
    static constexpr int kQueries = RT * (D / 16) * 512, kWeights = RT * kWarps * 512;  // bytes
    static constexpr int kSmem = kStages * kStage + kQueries + kWeights;
    static constexpr int kNT = D / 8, kGroup = kNT * 128 + 32;  // floats of 16 rows of a part
    static_assert(kCtas * (kSmem + 1024 + 288 + 44 * kPlans + 20 * kRows + kStages * (kTile * 4 + 16)) <= 228 * 1024, "shared memory");
};

// One item of a CTA's share, as thread 0 plans it for all: the walk over the
// requests would take some 50 registers of every thread.
struct ItemPlan {
    Request rq;
    int b, h, row0, t0, t1;  // request, KV head, the item's first row, its tiles of this CTA
    int last;                // the last CTA with a part of the item (begun and not done)
    bool there, begun, done;
};

template <int D, int RT>
__global__ void __launch_bounds__(kThreads, (SplitCfg<D, RT>::kCtas)) attention_split_kernel(const __grid_constant__ AttnParams p)
{
    using C = SplitCfg<D, RT>;
    static_assert(RT * 16 * 4 <= 1024 && kTile == 16 * kWarps, "a key group per warp");
    __shared__ uint32_t page_scales[C::kStages][kTile];  // bf16 bits of 2^ek and 2^-ev
    __shared__ float4 tops[C::kRows];  // per row, the warps' maxima; at the end their sums
    __shared__ float row_scales[C::kRows];
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t scratch[kWarps + 4];
    __shared__ uint32_t live[C::kStages][kWarps];
    __shared__ int any_bad;
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2;
    const uint32_t stages = saddr(smem), queries = stages + C::kStages * C::kStage, weights = queries + C::kQueries;
    unsigned flags = 0;
    const int mask_limit = p.mask_kind == 2 ? 64 * p.mask_words : 0x7fffffff;

    // ---- this CTA's share of the units
    const int ctas = gridDim.x, cta = blockIdx.x;
    using W = Walk<C::kRows, kTile, kItemCost>;
    auto sharing = [&](int64_t total) { return (int)min((int64_t)ctas, max((int64_t)(ctas / C::kCtas), total / kGrain)); };
    const Find f = find_request<kThreads>(p.num_requests, scratch, [&](int b) { return W::units(p, request(p, b, mask_limit, flags)); },
                                          sharing);
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
    // ---- thread 0 plans the items
    __shared__ W walk;
    __shared__ int64_t units;
    __shared__ ItemPlan plan[C::kPlans];
    auto plan_next = [&](int item) {
        ItemPlan &to = plan[item & (C::kPlans - 1)];
        to.there = walk.more();
        if (!to.there)
            return;
        to.rq = walk.rq, to.b = walk.b, to.h = walk.head(), to.row0 = walk.row0(), to.t0 = walk.t0, to.t1 = walk.t1;
        to.begun = walk.begun(), to.done = walk.finished();
        to.last = to.begun && !to.done ? walk.last_cta(Shares(units, sharing(units))) : 0;
        walk.next(p);
    };
    // copies run kStages - 1 tiles ahead, the block table's entries a tile more, plans an item more
    static_assert(C::kStages + 2 <= C::kPlans, "plans in use");
    int planned = C::kStages;  // the last item planned
    if (tid == 0) {
        const Shares shares(f.total, sharing(f.total));
        units = f.total;
        walk.start(p, shares.start(cta), shares.start(cta + 1), f.b, f.before, mask_limit);
        for (int i = 0; i <= planned; i++)
            plan_next(i);
    }
    __syncthreads();

    Loader<C::kRow> ld;
    // the tile that is copied next: `of` of its item (end: no more)
    struct {
        int item, tile, end, b, h, len;
    } to;
    auto enter = [&](int item) {
        const ItemPlan &i = plan[item & (C::kPlans - 1)];
        to.item = item, to.tile = i.t0, to.end = i.there ? i.t1 : -1, to.b = i.b, to.h = i.h, to.len = i.rq.ctx + i.rq.nq;
    };
    enter(0);
    auto fetch = [&]() {
        if (to.end >= 0)
            ld.fetch(p, to.b, to.tile, to.len);
    };
    auto issue = [&](int stage) {
        ld.store_scales();
        if (to.end >= 0) {
            ld.load(p, to.h, stages + stage * C::kStage, live[stage], flags);
            ld.fetch_scales(p, to.h, page_scales[stage]);
            if (++to.tile >= to.end)
                enter(to.item + 1);
            fetch();
        }
        cp_commit();
    };
    fetch();
#pragma unroll
    for (int s = 0; s < C::kStages - 1; s++)
        issue(s);

    float o[RT][2 * C::kWords][4], m[RT][2], l[RT][2];
    // o += the weights times V of the tile in `st`, this warp's dims
    auto add_v = [&](uint32_t st) {
#pragma unroll
        for (int jj = 0; jj < kWarps; jj += 2) {  // 32 keys
            uint32_t a[RT][4];
            auto load = [&](int k) {
#pragma unroll
                for (int t = 0; t < RT; t++)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(a[t][0]), "=r"(a[t][1]), "=r"(a[t][2]), "=r"(a[t][3])
                                 : "r"(weights + ((t * kWarps + jj + k) * 32 + lane) * 16)
                                 : "memory");
            };
            // word i of this warp's and 16 keys: the operands of the even and of the odd dims
            auto product = [&](uint32_t lo, uint32_t hi, int i) {
                const uint32_t x0 = __byte_perm(lo, 0, 0x3120), x1 = __byte_perm(hi, 0, 0x3120);
                const uint32_t e0 = e4m3_to_half2((uint16_t)x0), e1 = e4m3_to_half2((uint16_t)x1);
                const uint32_t q0 = e4m3_to_half2((uint16_t)(x0 >> 16)), q1 = e4m3_to_half2((uint16_t)(x1 >> 16));
#pragma unroll
                for (int t = 0; t < RT; t++) {
                    mma<true>(o[t][2 * i], a[t], e0, e1);
                    mma<true>(o[t][2 * i + 1], a[t], q0, q1);
                }
            };
            if constexpr (C::kWords == 1) {
                const int x = 16 * jj + lane;
                uint32_t v[4];
                ldsm4t(v, st + x * C::kRow + (((D / 16 + warp) ^ swz(x)) << 4));
                load(0);
                product(v[0], v[1], 0);
                load(1);
                product(v[2], v[3], 0);
            } else {
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    load(k);
#pragma unroll
                    for (int i = 0; i < C::kWords; i += 2) {
                        const int x = 16 * (jj + k) + (lane & 15);
                        uint32_t v[4];
                        ldsm4t(v, st + x * C::kRow + (((D / 16 + C::kWords * warp + i + (lane >> 4)) ^ swz(x)) << 4));
                        product(v[0], v[1], i);
                        product(v[2], v[3], i + 1);
                    }
                }
            }
        }
    };

    int stage = 0, item = 0, tile = plan[0].t0, end = plan[0].t1, ctx = plan[0].rq.ctx, len = ctx + plan[0].rq.nq;
    bool first = true;
    while (plan[item & (C::kPlans - 1)].there) {
        const ItemPlan &now = plan[item & (C::kPlans - 1)];
        if (first) {
            if (warp < RT) {  // behind the barrier that ends the item before
                uint32_t qa[D / 16][4];
                float rs[2];
                load_q<D, true>(p, now.rq, now.h, now.row0 + 16 * warp, qa, rs);
#pragma unroll
                for (int k = 0; k < D / 16; k++)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(queries + ((warp * (D / 16) + k) * 32 + lane) * 16),
                                 "r"(qa[k][0]), "r"(qa[k][1]), "r"(qa[k][2]), "r"(qa[k][3])
                                 : "memory");
                if ((lane & 3) == 0)
                    row_scales[16 * warp + g] = p.scale * kLog2e * rs[0], row_scales[16 * warp + 8 + g] = p.scale * kLog2e * rs[1];
            }
#pragma unroll
            for (int t = 0; t < RT; t++) {
#pragma unroll
                for (int n = 0; n < 2 * C::kWords; n++)
                    o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.0f;
                m[t][0] = m[t][1] = kNothing, l[t][0] = l[t][1] = 0.0f;
            }
            if (tid == 0)
                any_bad = 0;
        }
        cp_wait<C::kStages - 2>();
        __syncthreads();  // the tile has landed for all, the weights of the one before are written
        const uint32_t st = stages + stage * C::kStage;
        const int key0 = tile * kTile;
        const bool drafted = key0 + kTile > ctx;  // the tile holds drafted tokens or ends beyond them
        if (drafted) {
            if (zero_nonfinite<true, C::kRow>(smem + stage * C::kStage, ctx - key0, len - key0))
                any_bad = 1;
            __syncthreads();
        }
        if (planned == to.item) {
            planned++;
            if (tid == 0)
                plan_next(planned);
        }
        // ---- the scores of this warp's 16 keys
        float s[RT][2][4];
#pragma unroll
        for (int t = 0; t < RT; t++)
#pragma unroll
            for (int n = 0; n < 2; n++)
                s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.0f;
#pragma unroll
        for (int u = 0; u < D / 64; u++) {
            uint32_t x[2][4];
#pragma unroll
            for (int n = 0; n < 2; n++) {
                const int y = 16 * warp + 8 * n + g;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x[n][0]), "=r"(x[n][1]), "=r"(x[n][2]), "=r"(x[n][3])
                             : "r"(st + y * C::kRow + (((4 * u + (lane & 3)) ^ swz(y)) << 4))
                             : "memory");
            }
#pragma unroll
            for (int k = 0; k < 4; k++) {
                uint32_t k0[2], k1[2];
#pragma unroll
                for (int n = 0; n < 2; n++)
                    k0[n] = e4m3_to_half2((uint16_t)x[n][k]), k1[n] = e4m3_to_half2((uint16_t)(x[n][k] >> 16));
#pragma unroll
                for (int t = 0; t < RT; t++) {
                    uint32_t a[4];
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                                 : "r"(queries + ((t * (D / 16) + 4 * u + k) * 32 + lane) * 16)
                                 : "memory");
                    mma<true>(s[t][0], a, k0[0], k1[0]);
                    mma<true>(s[t][1], a, k0[1], k1[1]);
                }
            }
        }
        const uint32_t lv = live[stage][warp];
        float back[2][2];  // 2^-ev of this lane's keys
#pragma unroll
        for (int n = 0; n < 2; n++) {
            const uint2 v = *reinterpret_cast<const uint2 *>(&page_scales[stage][16 * warp + 8 * n + 2 * (lane & 3)]);
            const float k0 = __uint_as_float(v.x << 16), k1 = __uint_as_float(v.y << 16);
            // ev = 127 - the exponent's bits, through the last place of 2^23 + x
            const float e0 = 8388735.0f - __uint_as_float(0x4b000000u | v.x >> 23), e1 = 8388735.0f - __uint_as_float(0x4b000000u | v.y >> 23);
            back[n][0] = __uint_as_float(v.x & 0xffff0000u), back[n][1] = __uint_as_float(v.y & 0xffff0000u);
#pragma unroll
            for (int t = 0; t < RT; t++) {
                float(&x)[4] = s[t][n];
                const float c0 = row_scales[16 * t + g], c1 = row_scales[16 * t + 8 + g];
                x[0] = fmaf(x[0], c0 * k0, e0), x[1] = fmaf(x[1], c0 * k1, e1);
                x[2] = fmaf(x[2], c1 * k0, e0), x[3] = fmaf(x[3], c1 * k1, e1);
            }
        }
        if (drafted || lv != 0xffffu) {
#pragma unroll
            for (int t = 0; t < RT; t++) {
                const int r = now.row0 + 16 * t + g, i0 = r / p.group, i1 = (r + 8) / p.group, rows = now.rq.nq * p.group;
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int y = 8 * n + 2 * (lane & 3) + e, a = key0 + 16 * warp + y - now.rq.ctx;
                        const bool in = (lv >> y) & 1u;
                        if (!in || !(r < rows && sees(p, now.rq, i0, a)))
                            s[t][n][e] = -INFINITY;
                        if (!in || !(r + 8 < rows && sees(p, now.rq, i1, a)))
                            s[t][n][2 + e] = -INFINITY;
                    }
            }
        }
#pragma unroll
        for (int t = 0; t < RT; t++) {
            float t0 = fmaxf(fmaxf(s[t][0][0], s[t][0][1]), fmaxf(s[t][1][0], s[t][1][1]));
            float t1 = fmaxf(fmaxf(s[t][0][2], s[t][0][3]), fmaxf(s[t][1][2], s[t][1][3]));
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
            if ((lane & 3) == 0) {
                reinterpret_cast<float *>(&tops[16 * t + g])[warp] = t0;
                reinterpret_cast<float *>(&tops[16 * t + 8 + g])[warp] = t1;
            }
        }
        if (!first)
            add_v(stages + (stage == 0 ? C::kStages - 1 : stage - 1) * C::kStage);
        __syncthreads();  // the maxima and plans are there; the tile before and its weights are done with
        issue(stage == 0 ? C::kStages - 1 : stage - 1);
        float top[RT][2];
        bool grown = false;
#pragma unroll
        for (int t = 0; t < RT; t++)
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const float4 v = tops[16 * t + 8 * x + g];
                top[t][x] = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
                grown |= top[t][x] - m[t][x] > kLimit;
            }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int t = 0; t < RT; t++) {
                float f[2];
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    const float to = top[t][x] - m[t][x] > kLimit ? reference_of<true>(top[t][x]) : m[t][x];
                    f[x] = ex2(m[t][x] - to);
                    m[t][x] = to;
                    l[t][x] *= f[x];
                }
#pragma unroll
                for (int n = 0; n < 2 * C::kWords; n++)
                    o[t][n][0] *= f[0], o[t][n][1] *= f[0], o[t][n][2] *= f[1], o[t][n][3] *= f[1];
            }
        }
#pragma unroll
        for (int t = 0; t < RT; t++) {
#pragma unroll
            for (int n = 0; n < 2; n++) {
                float(&x)[4] = s[t][n];
                x[0] = ex2(x[0] - m[t][0]), x[1] = ex2(x[1] - m[t][0]);
                x[2] = ex2(x[2] - m[t][1]), x[3] = ex2(x[3] - m[t][1]);
                // this lane's columns; joined at the end
                l[t][0] = fmaf(x[1], back[n][1], fmaf(x[0], back[n][0], l[t][0]));
                l[t][1] = fmaf(x[3], back[n][1], fmaf(x[2], back[n][0], l[t][1]));
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(weights + ((t * kWarps + warp) * 32 + lane) * 16),
                         "r"(pack2<true>(s[t][0][0], s[t][0][1])), "r"(pack2<true>(s[t][0][2], s[t][0][3])),
                         "r"(pack2<true>(s[t][1][0], s[t][1][1])), "r"(pack2<true>(s[t][1][2], s[t][1][3]))
                         : "memory");
        }
        stage = stage + 1 == C::kStages ? 0 : stage + 1;
        first = false;
        if (++tile < end)
            continue;
        __syncthreads();  // the last tile's weights are written, the maxima read
        add_v(st);
        const Request rq = now.rq;
        const int h = now.h, row0 = now.row0, b = now.b, rows = rq.nq * p.group;

        // ---------------------------------------------------------------- the item ends here, or the CTA's share does
#pragma unroll
        for (int t = 0; t < RT; t++)
#pragma unroll
            for (int x = 0; x < 2; x++) {
                l[t][x] += __shfl_xor_sync(0xffffffffu, l[t][x], 1);
                l[t][x] += __shfl_xor_sync(0xffffffffu, l[t][x], 2);
                if ((lane & 3) == 0)
                    reinterpret_cast<float *>(&tops[16 * t + 8 * x + g])[warp] = l[t][x];
            }
        __syncthreads();
        const bool begun = now.begun, done = now.done;
        const int bad = any_bad;
#pragma unroll
        for (int t = 0; t < RT; t++) {
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const float4 v = tops[16 * t + 8 * x + g];
                l[t][x] = (v.x + v.y) + (v.z + v.w);
            }
            if (begun && done) {
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    const int r = row0 + 16 * t + 8 * x + g;
                    if (r >= rows)
                        continue;
                    const int i = r / p.group, hq = h * p.group + (r - i * p.group);
                    const int64_t at = (int64_t)(rq.q0 + i) * p.num_heads + hq;
                    const float sum = l[t][x], inv = sum > 0.0f ? 1.0f / sum : sum;  // (0: nothing seen; NaN stays)
                    if (warp == 0 && (lane & 3) == 0)
                        p.lse[at] = sum == 0.0f ? -INFINITY : m[t][x] * kLn2 + logf(sum);
                    uint16_t *dst = p.out + at * D + 16 * C::kWords * warp + 4 * (lane & 3);
#pragma unroll
                    for (int k = 0; k < C::kWords; k++)  // dims 16 k + 4 t ...: even tile, odd tile, even, odd
                        *reinterpret_cast<uint2 *>(dst + 16 * k) =
                            make_uint2(pack_bf16x2(o[t][2 * k][2 * x] * inv, o[t][2 * k + 1][2 * x] * inv),
                                       pack_bf16x2(o[t][2 * k][2 * x + 1] * inv, o[t][2 * k + 1][2 * x + 1] * inv));
                }
            } else {
                float *part = parts + (((int64_t)cta * 2 + (begun ? 1 : 0)) * RT + t) * C::kGroup;
#pragma unroll
                for (int n = 0; n < 2 * C::kWords; n++)
#pragma unroll
                    for (int x = 0; x < 4; x++)
                        part[((2 * C::kWords * warp + n) * 4 + x) * 32 + lane] = o[t][n][x];
                if (warp == 0 && (lane & 3) == 0) {
                    part[C::kNT * 128 + g] = m[t][0], part[C::kNT * 128 + 8 + g] = m[t][1];
                    part[C::kNT * 128 + 16 + g] = l[t][0], part[C::kNT * 128 + 24 + g] = l[t][1];
                }
            }
        }
        if (bad && begun && done) {
            __syncwarp();  // the warp's dims of the rows are written: a lane a row adds to them
            for (int x = lane; x < C::kRows && row0 + x < rows; x += 32) {
                const int r = row0 + x, i = r / p.group;
                add_nonfinite<D, true>(p, b, rq, h, i, p.out + ((int64_t)(rq.q0 + i) * p.num_heads + h * p.group + (r - i * p.group)) * D,
                                       16 * C::kWords * warp, 16 * C::kWords * (warp + 1));
            }
            __syncwarp();
        }
        if (begun && !done && tid == 0) {
            PartDesc &d = descs[cta];
            d.q0 = rq.q0, d.rows = rows, d.row0 = row0, d.h = h, d.nq = rq.nq, d.ctx = rq.ctx, d.b = b;
            d.last = now.last;
        }
        if (bad && !(begun && done) && tid == 0)
            descs[cta].bad[begun ? 1 : 0] = 1;
        {
            const ItemPlan &next = plan[++item & (C::kPlans - 1)];
            tile = next.t0, end = next.t1, ctx = next.rq.ctx, len = ctx + next.rq.nq;
            first = true;
        }
        __syncthreads();  // any_bad, the queries and the sums are free again
    }
    cp_wait<0>();
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && lane == 0 && p.error_flags)
        atomicOr(p.error_flags, flags);
}

template <int D, int RT>
cudaError_t split_ctas(int &ctas)
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
        using C = SplitCfg<D, RT>;
        e = prepare(attention_split_kernel<D, RT>, C::kSmem, C::kCtas, have);
        if (e != cudaSuccess)
            return e;
        __atomic_store_n(&cached[dev], have, __ATOMIC_RELEASE);
    }
    ctas = have;
    return cudaSuccess;
}

template <int D, int RT>
cudaError_t attention_split(const AttnParams &p, cudaStream_t stream)
{
    using C = SplitCfg<D, RT>;
    int ctas = 0;
    cudaError_t e = split_ctas<D, RT>(ctas);
    // Four CTAs that take every register of an SM are not launched early: placed between those
    // that the kernel before still has there, some find no slot (of 608 eight began when others
    // had ended).  64 requests, us, early / not: D 64, 8 rows 118 / 83 (95 / 85 behind an insert),
    // 32 rows 130 / 107, D 128, 8 rows 144 / 107.  With fewer CTAs early is as good or better (56
    // rows of D 128 235 / 238); what it costs four is 0.2 us of a request over 300 tokens (9.5).
    if (e == cudaSuccess)
        e = C::kCtas == 4 ? launch_whole(attention_split_kernel<D, RT>, ctas, kThreads, C::kSmem, stream, p)
                          : launch_pdl(attention_split_kernel<D, RT>, ctas, kThreads, C::kSmem, stream, p);
    if (e != cudaSuccess)
        return e;
    return launch_pdl_grid(join_kernel<D, true, RT>, dim3((unsigned)ctas, (unsigned)RT), kThreads, 0, 0, stream, p, ctas);
}

template <int D>
int64_t workspace_scaled_d(int wr, cudaError_t &e)
{
    int ctas = 0;
    e = wr == 1 ? split_ctas<D, 1>(ctas) : wr == 2 ? split_ctas<D, 2>(ctas) : split_ctas<D, 4>(ctas);
    return e == cudaSuccess ? (int64_t)ctas * ((int64_t)sizeof(PartDesc) + 2 * (int64_t)wr * Cfg<D, true, 1>::kPart * 4) : 0;
}

template <int D>
cudaError_t attention_scaled_d(const AttnParams &p, int wr, cudaStream_t stream)
{
    return wr == 1 ? attention_split<D, 1>(p, stream) : wr == 2 ? attention_split<D, 2>(p, stream) : attention_split<D, 4>(p, stream);
}

}  // namespace attn
}  // namespace dspark
