// The drafted tokens' attention on the 5th-generation tensor cores, for
// requests of more than a few query rows (tcgen05 + tensor memory, sm_103a).
// Mathematics, rows, items, splitting and masking as in tree_attn_mma.cuh.
//
// Why.  With r rows of queries a cached token of D 128 brings 512 bytes and
// 512 r flops: the card's rates balance at r = 283, but mma.sync, whose
// operands pass through registers, was bound by issue from r = 56 on (64
// requests x 7 tokens x 8 heads: 234 us against 136 us of memory time).
//
// One CTA per SM, an item is up to 256 rows of a (request, KV head), a tile
// 128 keys.  Two streams of softmax (a warpgroup each, a thread per query
// row, no shuffles) keep the tensor cores busy: with more than 128 rows a
// stream is a half of the rows and every tile serves both; with up to 128
// the streams share the rows and take every other tile, their results joined
// in the end.  Tensor memory: scores S of both streams (128 fp32 columns
// each, overwritten by the weights P, two 16-bit values a column, which feed
// the second product from there) and both outputs (D columns each).
//
//  - producer warps (4): gather the tile's K and V through the block table
//    into separate rings, bf16 with 16-byte asynchronous copies straight into
//    the operands' 128-byte swizzle, fp8 through registers, converted to
//    fp16 once per tile instead of once per row tile;
//  - one thread issues S = Q K^T (depth D) and O += P V (V as the cache holds
//    it: its N direction contiguous), in the order S0 S1 | PV0 S0' PV1 S1' |
//    so that one stream's products run under the other's softmax;
//  - softmax warps (8): 64 scores of a row at a time in registers, maximum,
//    base-2 exponentials with paired fp32 instructions, P back to tensor
//    memory.  The output is rescaled only when a row's maximum has grown by
//    more than 2^8 since the value in use: until then the weights exceed 1,
//    which costs neither range nor precision.
//
// 13 warps leave 128 registers a thread, so a row's 128 scores are read twice
// (for the maximum and for the weights), 64 at a time.
// Every wait is bounded; on expiry the CTA raises DSPARK_FLAG_TIMEOUT, stops
// issuing, waits for its copies and products in flight, frees its tensor
// memory and returns.
#pragma once

#include <type_traits>

#include "tc_ptx.cuh"
#include "tree_attn_mma.cuh"

namespace dspark {
namespace attn {

constexpr int kTcThreads = 416, kKeysTc = 128;  // 8 softmax warps, 4 producers, 1 that issues the products
constexpr float kLazy = 8.0f;  // growth of a maximum (log2) that waits for a rescale

template <int D, bool FP8>
struct TcCfg {
    static constexpr int kStages = D == 64 ? 4 : 2;       // of the K ring and of the V ring
    static constexpr int kTileBytes = kKeysTc * D * 2;    // one K or V tile, 16-bit
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kRow = 2 * D * (FP8 ? 1 : 2);    // bytes of a cached token
    static constexpr int kSmem = 1024 + 2 * kQBytes + 2 * kStages * kTileBytes;
    static constexpr int kRowPart = (D + 2) * 128;        // floats of one row tile's part
    static constexpr int kPart = 2 * kRowPart;
};

template <int D, bool FP8>
__global__ void __launch_bounds__(kTcThreads, 1) attention_tc_kernel(const __grid_constant__ AttnParams p)
{
    using C = TcCfg<D, FP8>;
    using namespace tc;
    constexpr int NS = C::kStages;
    constexpr uint32_t kS[2] = {0, 128}, kO[2] = {256, 256 + 128};  // tensor-memory columns
    constexpr uint32_t kIdQK = idesc(FP8, false, 128, kKeysTc), kIdPV = idesc(FP8, true, 128, D);
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (tc::saddr(smem_raw) & 1023u)) & 1023u);
    unsigned char *sq = smem, *sk = smem + 2 * C::kQBytes, *sv = sk + NS * C::kTileBytes;
    __shared__ uint64_t kfull[NS], kempty[NS], vfull[NS], vempty[NS], qfull[2], sfull[2], pfull[2], ofull[2], jfull, jempty, done;
    __shared__ uint32_t tmem_slot, live[8][4];
    __shared__ int abort_flag, bad[16];
    __shared__ float join_ml[256];
    __shared__ int64_t scratch[kTcThreads / 32 + 4];
    volatile int *abort = &abort_flag;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < NS; s++) {
            bar_init(kfull + s, 128 + 4);  // the producers' copies, and their live masks
            bar_init(vfull + s, 128);
            bar_init(kempty + s, 1);
            bar_init(vempty + s, 1);
        }
        for (int s = 0; s < 2; s++) {
            bar_init(qfull + s, 128);
            bar_init(pfull + s, 4);
            bar_init(sfull + s, 1);
            bar_init(ofull + s, 1);
        }
        bar_init(&jfull, 128);
        bar_init(&jempty, 128);
        bar_init(&done, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::saddr(&tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_enter();
    unsigned flags = 0;
    const int mask_limit = p.mask_kind == 2 ? 64 * p.mask_words : 0x7fffffff;

    // ---- this CTA's share of the units
    const int ctas = gridDim.x, cta = blockIdx.x;
    const Find f = find_request<kTcThreads>(
        p.num_requests, scratch,
        [&](int b) -> int64_t {
            const Request r = request(p, b, mask_limit, flags);
            if (r.nq == 0)
                return 0;
            const int64_t items = (int64_t)p.num_kv_heads * (((int64_t)r.nq * p.group + 255) / 256);
            return items * ((r.ctx + r.nq + kKeysTc - 1) / kKeysTc);
        },
        [&](int64_t total) -> int64_t {
            const int64_t n = total < ctas ? total : ctas;
            return cta < n ? (int64_t)((unsigned long long)total * cta / (unsigned long long)n) : -1;
        });
    const int64_t total = f.total, n_cta = total < ctas ? total : ctas;
    PartDesc *descs = reinterpret_cast<PartDesc *>(p.parts);
    float *parts = p.parts + (int64_t)ctas * (sizeof(PartDesc) / 4);
    if (tid == 0)
        descs[cta].last = -1, descs[cta].bad[0] = 0, descs[cta].bad[1] = 0;
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;
    int64_t lo = 0, hi = 0;
    if (f.b >= 0) {
        lo = (int64_t)((unsigned long long)total * cta / (unsigned long long)n_cta);
        hi = (int64_t)((unsigned long long)total * (cta + 1) / (unsigned long long)n_cta);
    }

    // every role walks the CTA's units on its own, item by item
    struct Walk {
        int64_t u;
        int b, item, items, tile, tiles, rgs;
        Request rq;
    };
    auto enter = [&](Walk &w) {
        unsigned ignore = 0;
        w.rq = request(p, w.b, mask_limit, ignore);
        w.rgs = (w.rq.nq * p.group + 255) / 256;
        w.items = w.rq.nq ? p.num_kv_heads * w.rgs : 0;
        w.tiles = (w.rq.ctx + w.rq.nq + kKeysTc - 1) / kKeysTc;
    };
    auto start = [&]() {
        Walk w;
        w.u = lo;
        w.b = f.b;
        w.item = w.tile = 0;
        w.tiles = 1;
        if (lo < hi) {
            enter(w);
            const int64_t in = lo - f.before;
            w.item = (int)(in / w.tiles);
            w.tile = (int)(in - (int64_t)w.item * w.tiles);
        }
        return w;
    };
    // the tiles of the item at w that are this CTA's
    auto share = [&](const Walk &w) { return (int)min((int64_t)(w.tiles - w.tile), hi - w.u); };
    auto next = [&](Walk &w, int n) {  // past those tiles
        w.u += n;
        w.tile = 0;
        if (w.u < hi && ++w.item >= w.items) {
            w.item = 0;
            do {
                w.b++;
                enter(w);
            } while (w.items == 0);
        }
    };

    if (warp >= 12) {
        // ------------------------------------------------------------ the issuing thread
        if (tid == 12 * 32) {
            Walk w = start();
            int base = 0;            // tiles consumed before this item
            int nq[2] = {0, 0};      // Q tiles used
            int np[2] = {0, 0};      // P tiles used
            bool ok = true;
            while (w.u < hi && ok) {
                const int n = share(w);
                const int row0 = (w.item % w.rgs) * 256;
                const bool two = w.rq.nq * p.group - row0 > 128;
                auto qk = [&](int s, int j, bool last) {
                    const int x = base + j, st = x % NS;
                    if (!ok || !bar_wait(kfull + st, (uint32_t)(x / NS) & 1u, abort)) {
                        ok = false;
                        return;
                    }
                    fence_async();
                    fence_after();
                    const uint32_t a = tc::saddr(sq + (two ? s : 0) * C::kQBytes), b = tc::saddr(sk + st * C::kTileBytes);
#pragma unroll
                    for (int k = 0; k < D / 16; k++)
                        mma_ss(tmem + kS[s], desc128(a + (k / 4) * 16384 + (k % 4) * 32, 16),
                               desc128(b + (k / 4) * 16384 + (k % 4) * 32, 16), kIdQK, k != 0);
                    mma_commit(sfull + s);
                    if (last)
                        mma_commit(kempty + st);
                };
                auto pv = [&](int s, int j, bool first, bool last) {
                    const int x = base + j, st = x % NS;
                    if (!ok || !bar_wait(vfull + st, (uint32_t)(x / NS) & 1u, abort) ||
                        !bar_wait(pfull + s, (uint32_t)np[s] & 1u, abort)) {
                        ok = false;
                        return;
                    }
                    np[s]++;
                    fence_async();
                    fence_after();
                    const uint32_t b = tc::saddr(sv + st * C::kTileBytes);
#pragma unroll
                    for (int k = 0; k < kKeysTc / 16; k++)
                        mma_ts(tmem + kO[s], tmem + kS[s] + 8 * k, desc128(b + k * 2048, 16384), kIdPV, !(first && k == 0));
                    mma_commit(ofull + s);
                    if (last)
                        mma_commit(vempty + st);
                };
                for (int s = 0; s < (two ? 2 : 1) && ok; s++)
                    ok = bar_wait(qfull + s, (uint32_t)(nq[s]++) & 1u, abort);
                qk(0, 0, !two);
                if (two)
                    qk(1, 0, true);
                else if (n > 1)
                    qk(1, 1, true);
                for (int j = 0; j < n && ok; j++) {
                    if (two) {
                        pv(0, j, j == 0, false);
                        if (j + 1 < n)
                            qk(0, j + 1, false);
                        pv(1, j, j == 0, true);
                        if (j + 1 < n)
                            qk(1, j + 1, true);
                    } else {
                        pv(j & 1, j, j < 2, true);
                        if (j + 2 < n)
                            qk(j & 1, j + 2, true);
                    }
                }
                base += n;
                next(w, n);
            }
            mma_commit(&done);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ------------------------------------------------------------ producers: a thread per tile row for the addresses
        const int pw = warp - 8;
        Walk w = start();
        int base = 0, item_no = 0;
        bool ok = true;
        int64_t phys = 0;
        int off = 0;
        bool in = false;
        auto fetch = [&](int b, int tile, int len) {
            const int j = tile * kKeysTc + pw * 32 + lane;
            in = j < len;
            phys = 0, off = 0;
            if (in) {
                const int blk = j / p.block_size;
                off = j - blk * p.block_size;
                phys = __ldg(p.table + b * p.table_stride + blk);
            }
        };
        if (w.u < hi)
            fetch(w.b, w.tile, w.rq.ctx + w.rq.nq);
        while (w.u < hi && ok) {
            const int n = share(w), len = w.rq.ctx + w.rq.nq, ctx = w.rq.ctx, tile0 = w.tile;
            const int h = w.item / w.rgs;
            Walk after = w;
            next(after, n);
            if (tid == 8 * 32)
                bad[item_no & 15] = 0;
            for (int j = 0; j < n; j++) {
                const int x = base + j, st = x % NS;
                const uint32_t parity = ((uint32_t)(x / NS) & 1u) ^ 1u;
                bool here = in;
                if (here && (phys < 0 || phys >= p.num_blocks)) {
                    flags |= kFlagBlockRange;
                    here = false;
                }
                const unsigned bits = __ballot_sync(0xffffffffu, here);
                const unsigned long long row = reinterpret_cast<unsigned long long>(
                    p.cache + (here ? ((phys * p.num_kv_heads + h) * p.block_size + off) * (int64_t)C::kRow : 0));
                // the next tile's blocks
                if (j + 1 < n)
                    fetch(w.b, tile0 + j + 1, len);
                else if (after.u < hi)
                    fetch(after.b, after.tile, after.rq.ctx + after.rq.nq);
                const int key0 = (tile0 + j) * kKeysTc;
                const bool drafted = key0 + kKeysTc > ctx;
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    uint64_t *full = half ? vfull + st : kfull + st, *empty = half ? vempty + st : kempty + st;
                    const uint32_t dst0 = tc::saddr((half ? sv : sk) + st * C::kTileBytes);
                    if constexpr (FP8) {
                        constexpr int kW = D / 16, kIt = kW;  // 16-byte words of a row's half; 32 rows x kW words / 32 lanes
                        uint4 v[kIt];
#pragma unroll
                        for (int i = 0; i < kIt; i++) {
                            const int idx = i * 32 + lane, y = idx / kW, c = idx % kW;
                            const unsigned long long src = __shfl_sync(0xffffffffu, row, y);
                            v[i] = make_uint4(0, 0, 0, 0);
                            if ((bits >> y) & 1u)
                                v[i] = __ldg(reinterpret_cast<const uint4 *>(src + half * D + 16 * c));
                        }
                        ok = ok && bar_wait(empty, parity, abort);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok)
                            break;
#pragma unroll
                        for (int i = 0; i < kIt; i++) {
                            const int idx = i * 32 + lane, y = idx / kW, c = idx % kW, yy = pw * 32 + y;
                            uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                            if (half && drafted && key0 + yy >= ctx) {
#pragma unroll
                                for (int k = 0; k < 4; k++)
                                    if (nonfinite_word(q[k], true)) {
#pragma unroll
                                        for (int e = 0; e < 4; e++)
                                            if (((q[k] >> (8 * e)) & 0x7fu) == 0x7fu)
                                                q[k] &= ~(0xffu << (8 * e));
                                        bad[item_no & 15] = 1;
                                    }
                            }
                            uint32_t o[8];
#pragma unroll
                            for (int k = 0; k < 4; k++)
                                o[2 * k] = e4m3_to_half2((uint16_t)q[k]), o[2 * k + 1] = e4m3_to_half2((uint16_t)(q[k] >> 16));
#pragma unroll
                            for (int k = 0; k < 2; k++) {
                                const int cc = 2 * c + k;  // 16-byte word of the fp16 row
                                const uint32_t at = dst0 + (cc >> 3) * 16384 + yy * 128 + (((cc & 7) ^ (yy & 7)) << 4);
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(o[4 * k]), "r"(o[4 * k + 1]),
                                             "r"(o[4 * k + 2]), "r"(o[4 * k + 3])
                                             : "memory");
                            }
                        }
                        if (half == 0 && lane == 0)
                            live[x & 7][pw] = bits;
                        fence_async();
                        bar_arrive(full);
                        if (half == 0 && lane == 0)
                            bar_arrive(full);
                    } else {
                        constexpr int kW = D / 8, kIt = kW;
                        ok = ok && bar_wait(empty, parity, abort);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok)
                            break;
#pragma unroll
                        for (int i = 0; i < kIt; i++) {
                            const int idx = i * 32 + lane, y = idx / kW, c = idx % kW, yy = pw * 32 + y;
                            const unsigned long long src = __shfl_sync(0xffffffffu, row, y);
                            cp16(dst0 + (c >> 3) * 16384 + yy * 128 + (((c & 7) ^ (yy & 7)) << 4),
                                 reinterpret_cast<const unsigned char *>(src) + half * 2 * D + 16 * c, (bits >> y) & 1u);
                        }
                        if (half == 0 && lane == 0) {
                            live[x & 7][pw] = bits;
                            bar_arrive(full);
                        }
                        if (half && drafted) {
                            // infinities and NaN among the drafted V: zeroed here, accounted for at the end
                            asm volatile("cp.async.wait_all;" ::: "memory");
                            for (int i = 0; i < kIt; i++) {
                                const int idx = i * 32 + lane, y = idx / kW, c = idx % kW, yy = pw * 32 + y;
                                if (key0 + yy < ctx)
                                    continue;
                                uint4 *at = reinterpret_cast<uint4 *>(sv + st * C::kTileBytes + (c >> 3) * 16384 + yy * 128 +
                                                                      (((c & 7) ^ (yy & 7)) << 4));
                                const uint4 v = *at;
                                uint32_t q[4] = {v.x, v.y, v.z, v.w};
                                bool hit = false;
#pragma unroll
                                for (int k = 0; k < 4; k++)
                                    if (nonfinite_word(q[k], false)) {
                                        hit = true;
                                        if ((q[k] & 0x7f80u) == 0x7f80u)
                                            q[k] &= 0xffff0000u;
                                        if ((q[k] & 0x7f800000u) == 0x7f800000u)
                                            q[k] &= 0xffffu;
                                    }
                                if (hit) {
                                    *at = make_uint4(q[0], q[1], q[2], q[3]);
                                    bad[item_no & 15] = 1;
                                }
                            }
                            fence_async();
                            bar_arrive(full);
                        } else {
                            bar_arrive_copies(full);
                        }
                    }
                }
                if (!ok)
                    break;
            }
            base += n;
            item_no++;
            w = after;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ------------------------------------------------------------ softmax: a thread per query row
        const int s = warp >> 2, q4 = warp & 3, r = q4 * 32 + lane;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const float ks = FP8 && p.k_scale ? __ldg(p.k_scale) : 1.0f, vs = FP8 && p.v_scale ? __ldg(p.v_scale) : 1.0f;
        const float base_scale = p.scale * kLog2e * ks;
        Walk w = start();
        int base = 0, item_no = 0;
        int nS = 0, nO = 0;  // S tiles read, PV products issued (of this stream)
        int nJ = 0;          // items whose rows the streams shared
        bool ok = true;
        while (w.u < hi && ok) {
            const int n = share(w), rows = w.rq.nq * p.group;
            const int h = w.item / w.rgs, row0 = (w.item - h * w.rgs) * 256;
            const bool two = rows - row0 > 128;
            const int64_t item_start = w.u - w.tile;
            const bool begun = item_start >= lo, finished = item_start + w.tiles <= hi;
            const int rt = two ? s : 0, my = row0 + rt * 128 + r;
            const bool mine = my < rows, warp_live = row0 + rt * 128 + q4 * 32 < rows;
            const int i = mine ? my / p.group : 0, hq = h * p.group + (mine ? my - i * p.group : 0);
            const int steps = two ? n : s == 0 ? (n + 1) / 2 : n / 2;
            // ---- the query row.  A negative scale turns its sign, a zero one
            // zeroes it, so that the factor c of the scores is positive.
            float c = base_scale;
            if (two || s == 0 || FP8) {
                const uint16_t *src = p.q + (int64_t)(w.rq.q0 + i) * p.q_ts + (int64_t)hq * p.q_hs;
                const uint32_t flip = base_scale < 0.0f ? 0x80008000u : 0u;
                const bool zero = base_scale == 0.0f || !mine;
                const uint32_t dst0 = tc::saddr(sq + rt * C::kQBytes);
                float inv = 1.0f, fix = 1.0f;
                if constexpr (FP8) {
                    float top = 0.0f;
                    if (!zero)
#pragma unroll
                        for (int k = 0; k < D / 8; k++) {
                            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + k);
                            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(q[e] << 16)), fabsf(__uint_as_float(q[e] & 0xffff0000u))));
                        }
                    int e = 0;
                    if (top > 0.0f && top < __int_as_float(0x7f800000))
                        e = max(ilogbf(top), -126);
                    c *= scalbnf(1.0f, e);
                    inv = scalbnf(1.0f, e > 126 ? -126 : -e);
                    fix = e > 126 ? 0.5f : 1.0f;
                }
                if (two || s == 0) {
#pragma unroll
                    for (int k = 0; k < D / 8; k++) {
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (!zero)
                            v = __ldg(reinterpret_cast<const uint4 *>(src) + k);
                        uint32_t q[4] = {v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip};
                        if constexpr (FP8) {
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                q[e] = pack2<true>(__uint_as_float(q[e] << 16) * inv * fix, __uint_as_float(q[e] & 0xffff0000u) * inv * fix);
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst0 + (k >> 3) * 16384 + r * 128 + (((k & 7) ^ (r & 7)) << 4)),
                                     "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3])
                                     : "memory");
                    }
                    fence_async();
                    bar_arrive(qfull + rt);
                }
            }
            c = c == 0.0f ? 1.0f : fabsf(c);
            const uint64_t c2 = pr(c, c);
            float m = -INFINITY, l = 0.0f;  // the maximum in use (scaled, base 2), the sum of weights

            for (int k = 0; k < steps; k++) {
                const int j = two ? k : 2 * k + s;
                const int key0 = (w.tile + j) * kKeysTc;
                ok = ok && bar_wait(sfull + s, (uint32_t)nS & 1u, abort);
                nS++;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                fence_after();
                if (warp_live) {
                    const int lx = (base + j) & 7;
                    uint32_t vis[4] = {live[lx][0], live[lx][1], live[lx][2], live[lx][3]};  // bit b of vis[g]: key key0 + 32 g + b is seen
                    const bool drafted = key0 + kKeysTc > w.rq.ctx;
                    const bool masked = drafted || (vis[0] & vis[1] & vis[2] & vis[3]) != 0xffffffffu;
                    if (masked) {
                        const uint64_t *words = p.tree_mask + (int64_t)(w.rq.q0 + i) * p.mask_words;
                        const int limit = p.mask_kind == 1 ? min(w.rq.nq, i + 1) : w.rq.nq;
#pragma unroll
                        for (int g = 0; g < 4; g++) {
                            const int a0 = key0 + 32 * g - w.rq.ctx;  // the drafted token of bit 0; below 0: context
                            if (a0 > -32) {
                                const int sh = a0 < 0 ? -a0 : 0, a = a0 < 0 ? 0 : a0;  // bits below sh are context
                                uint32_t t = 0xffffffffu;
                                if (p.mask_kind == 2) {
                                    const int wd = a >> 6, bt = a & 63;
                                    uint64_t y = wd < p.mask_words ? __ldg(words + wd) >> bt : 0ull;
                                    if (bt > 32 && wd + 1 < p.mask_words)
                                        y |= __ldg(words + wd + 1) << (64 - bt);
                                    t = (uint32_t)y;
                                }
                                const int room = limit - a;
                                t = room <= 0 ? 0u : room < 32 ? t & ((1u << room) - 1u) : t;
                                vis[g] &= sh ? (t << sh) | ((1u << sh) - 1u) : t;
                            }
                            if (!mine)
                                vis[g] = 0;
                        }
                    }
                    // scores of half of the keys, -inf where not seen
                    auto load_half = [&](int half, uint32_t (&x)[64]) {
                        tmem_ld64(tmem + lanes + kS[s] + 64 * half, x);
                        if (masked) {
#pragma unroll
                            for (int e = 0; e < 64; e++)
                                if (!((vis[2 * half + (e >> 5)] >> (e & 31)) & 1u))
                                    x[e] = 0xff800000u;
                        }
                    };
                    // ---- maximum
                    float top = -INFINITY;
#pragma unroll
                    for (int half = 0; half < 2; half++) {
                        uint32_t x[64];
                        load_half(half, x);
                        float t0 = __uint_as_float(x[0]), t1 = __uint_as_float(x[1]), t2 = __uint_as_float(x[2]), t3 = __uint_as_float(x[3]);
#pragma unroll
                        for (int e = 4; e < 64; e += 4) {
                            t0 = fmaxf(t0, __uint_as_float(x[e])), t1 = fmaxf(t1, __uint_as_float(x[e + 1]));
                            t2 = fmaxf(t2, __uint_as_float(x[e + 2])), t3 = fmaxf(t3, __uint_as_float(x[e + 3]));
                        }
                        top = fmaxf(top, fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)));
                    }
                    const float t = top * c;
                    const bool grow = t > m + kLazy || (m == -INFINITY && t > m);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float old = m;
                        m = fmaxf(m, t);
                        const float fr = old == m ? 1.0f : ex2(old - m);  // 0 from -inf
                        l *= fr;
                        if (k > 0) {
                            // the products so far have to be in before they are rescaled
                            ok = ok && bar_wait(ofull + s, (uint32_t)(nO - 1) & 1u, abort);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok)
                                break;
                            fence_after();
#pragma unroll
                            for (int d = 0; d < D; d += 32) {
                                uint32_t o[32];
                                tmem_ld32(tmem + lanes + kO[s] + d, o);
#pragma unroll
                                for (int e = 0; e < 32; e++)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * fr);
                                tmem_st32(tmem + lanes + kO[s] + d, o);
                            }
                        }
                    }
                    const float mu = m == -INFINITY ? 0.0f : m;
                    const uint64_t m2 = pr(-mu, -mu);
                    uint64_t sum0 = 0, sum1 = 0;
                    // s c - m in one rounding; where m is so large that its own rounding
                    // shows in that (scores beyond 2^24), the product is rounded first
                    auto weights = [&](auto apart) {
#pragma unroll
                        for (int half = 0; half < 2; half++) {
                            uint32_t x[64], pk[32];
                            load_half(half, x);
#pragma unroll
                            for (int e = 0; e < 64; e += 4) {
                                const uint64_t x0 = pr(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                                const uint64_t x1 = pr(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                                float a0, a1, a2, a3;
                                if constexpr (decltype(apart)::value) {
                                    a0 = __fsub_rn(__fmul_rn(__uint_as_float(x[e]), c), mu), a1 = __fsub_rn(__fmul_rn(__uint_as_float(x[e + 1]), c), mu);
                                    a2 = __fsub_rn(__fmul_rn(__uint_as_float(x[e + 2]), c), mu), a3 = __fsub_rn(__fmul_rn(__uint_as_float(x[e + 3]), c), mu);
                                } else {
                                    unpr(fma2(x0, c2, m2), a0, a1);
                                    unpr(fma2(x1, c2, m2), a2, a3);
                                }
                                a0 = ex2(a0), a1 = ex2(a1), a2 = ex2(a2), a3 = ex2(a3);
                                sum0 = add2(sum0, pr(a0, a1));
                                sum1 = add2(sum1, pr(a2, a3));
                                pk[e / 2] = pack2<FP8>(a0, a1);
                                pk[e / 2 + 1] = pack2<FP8>(a2, a3);
                            }
                            // columns 32 half .. of P lie over scores that are used up
                            tmem_st32(tmem + lanes + kS[s] + 32 * half, pk);
                        }
                    };
                    if (__any_sync(0xffffffffu, fabsf(mu) > 16777216.0f))
                        weights(std::true_type{});
                    else
                        weights(std::false_type{});
                    float a0, a1;
                    unpr(add2(sum0, sum1), a0, a1);
                    l += a0 + a1;
                    tmem_wait_st();
                }
                fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(pfull + s);
                nO++;
            }
            if (!ok)
                break;
            // ---- the item ends here, or the CTA's share of it does
            if (steps > 0) {
                ok = bar_wait(ofull + s, (uint32_t)(nO - 1) & 1u, abort);
                ok = __all_sync(0xffffffffu, ok);
            }
            fence_after();
            float y0 = 1.0f, y1 = 0.0f;  // factors of the two streams' sums
            if (!two) {
                if (s == 1) {
                    join_ml[r] = m, join_ml[128 + r] = l;
                    fence_before();
                    bar_arrive(&jfull);
                    // its output and statistics stay until stream 0 has read them
                    ok = ok && bar_wait(&jempty, (uint32_t)nJ & 1u, abort);
                } else {
                    ok = ok && bar_wait(&jfull, (uint32_t)nJ & 1u, abort);
                    fence_after();
                    const float om = join_ml[r], ol = join_ml[128 + r], t = fmaxf(m, om), u = t == -INFINITY ? 0.0f : t;
                    y0 = ex2(m - u), y1 = ex2(om - u);
                    m = t;
                    l = l * y0 + ol * y1;
                }
                nJ++;
                ok = __all_sync(0xffffffffu, ok);
            }
            if (!ok)
                break;
            const int is_bad = bad[item_no & 15];
            if ((two || s == 0) && warp_live) {
                const bool other = !two && n > 1;
                float *part = parts + ((int64_t)cta * 2 + (begun ? 1 : 0)) * C::kPart + rt * C::kRowPart + r;
                const bool direct = begun && finished;
                const float inv = l > 0.0f ? vs / l : l == 0.0f ? 0.0f : l;
                const int64_t at = (int64_t)(w.rq.q0 + i) * p.num_heads + hq;
                uint16_t *dst = p.out + at * D;
#pragma unroll
                for (int d = 0; d < D; d += 32) {
                    uint32_t o[32];
                    tmem_ld32(tmem + lanes + kO[0 + (two ? s : 0)] + d, o);
                    if (other) {
                        uint32_t o1[32];
                        tmem_ld32(tmem + lanes + kO[1] + d, o1);
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * y0 + __uint_as_float(o1[e]) * y1);
                    }
                    if (!direct) {
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            part[(d + e) * 128] = __uint_as_float(o[e]);
                    } else if (mine) {
                        float v[32];
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            v[e] = __uint_as_float(o[e]) * inv;
                        if (is_bad) {
                            for (int a = 0; a < w.rq.nq; a++) {
                                if (!sees(p, w.rq, i, a))
                                    continue;
#pragma unroll
                                for (int e = 0; e < 32; e++) {
                                    const float z = drafted_v<D, FP8>(p, w.b, w.rq.ctx, h, a, d + e);
                                    if (!(fabsf(z) <= 3.4028235e38f))
                                        v[e] += z;
                                }
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4 *>(dst + d + e) =
                                make_uint4(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]), pack_bf16x2(v[e + 4], v[e + 5]),
                                           pack_bf16x2(v[e + 6], v[e + 7]));
                    }
                }
                if (!direct)
                    part[D * 128] = m, part[(D + 1) * 128] = l;
                else if (mine)
                    p.lse[at] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
            }
            fence_before();
            if (!two && s == 0)
                bar_arrive(&jempty);
            if (tid == 0) {
                if (begun && !finished) {
                    PartDesc &d = descs[cta];
                    d.q0 = w.rq.q0, d.rows = rows, d.row0 = row0, d.h = h, d.nq = w.rq.nq, d.ctx = w.rq.ctx, d.b = w.b;
                    d.last = (int32_t)(((unsigned long long)(item_start + w.tiles) * n_cta - 1) / (unsigned long long)total);
                }
                if (is_bad && !(begun && finished))
                    descs[cta].bad[begun ? 1 : 0] = 1;
            }
            base += n;
            item_no++;
            next(w, n);
        }
    }
    __syncthreads();
    if (warp == 12) {
        // every product has completed before the tensor memory is freed
        if (lane == 0) {
            const unsigned long long t0 = gtimer();
            while (!bar_try(&done, 0) && gtimer() - t0 < kTimeoutNs) {
            }
        }
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
    if (tid == 0 && *abort)
        flags |= kFlagTimeout;
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0 && flags && p.error_flags)
        atomicOr(p.error_flags, flags);
}

// Joins the parts of the item that CTA blockIdx.x began and did not finish:
// block y takes 32 dims (y % (D / 32)) of row tile y / (D / 32), a thread per row.
template <int D, bool FP8>
__global__ void __launch_bounds__(128) join_tc_kernel(const __grid_constant__ AttnParams p, int ctas)
{
    using C = TcCfg<D, FP8>;
    pdl_enter();
    const int r = threadIdx.x, rt = blockIdx.y / (D / 32), d0 = (blockIdx.y % (D / 32)) * 32;
    const PartDesc *descs = reinterpret_cast<const PartDesc *>(p.parts);
    const PartDesc d = descs[blockIdx.x];
    const int my = d.row0 + rt * 128 + r;
    if (d.last < 0 || my >= d.rows)
        return;
    const float *parts = p.parts + (int64_t)ctas * (sizeof(PartDesc) / 4);
    auto part = [&](int c) {
        return parts + ((int64_t)c * 2 + (c == (int)blockIdx.x ? 1 : 0)) * C::kPart + rt * C::kRowPart + r;
    };
    float m = -INFINITY;
    bool bad = d.bad[1] != 0;
    for (int c = blockIdx.x; c <= d.last; c++) {
        m = fmaxf(m, part(c)[D * 128]);
        if (c != (int)blockIdx.x)
            bad |= descs[c].bad[0] != 0;
    }
    const float u = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, o[32];
#pragma unroll
    for (int e = 0; e < 32; e++)
        o[e] = 0.0f;
    for (int c = blockIdx.x; c <= d.last; c++) {
        const float *at = part(c);
        const float x = ex2(at[D * 128] - u);
        l = fmaf(at[(D + 1) * 128], x, l);
#pragma unroll
        for (int e = 0; e < 32; e++)
            o[e] = fmaf(at[(d0 + e) * 128], x, o[e]);
    }
    const float vs = FP8 && p.v_scale ? __ldg(p.v_scale) : 1.0f;
    const float inv = l > 0.0f ? vs / l : l == 0.0f ? 0.0f : l;
    const int i = my / p.group, hq = d.h * p.group + (my - i * p.group);
    const int64_t at = (int64_t)(d.q0 + i) * p.num_heads + hq;
    if (d0 == 0)
        p.lse[at] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
    const Request rq{d.q0, d.nq, d.ctx};
#pragma unroll
    for (int e = 0; e < 32; e++) {
        o[e] *= inv;
        if (bad)
            o[e] += nonfinite_sum<D, FP8>(p, d.b, rq, d.h, i, d0 + e);
    }
#pragma unroll
    for (int e = 0; e < 32; e += 8)
        *reinterpret_cast<uint4 *>(p.out + at * D + d0 + e) =
            make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]), pack_bf16x2(o[e + 4], o[e + 5]),
                       pack_bf16x2(o[e + 6], o[e + 7]));
}

// ------------------------------------------------------------------ launches

template <int D, bool FP8>
cudaError_t attention_tc_ctas(int &ctas)
{
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
            e = cudaFuncSetAttribute(attention_tc_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcCfg<D, FP8>::kSmem);
        if (e != cudaSuccess)
            return e;
        __atomic_store_n(&cached[dev], have, __ATOMIC_RELEASE);
    }
    ctas = have;
    return cudaSuccess;
}

template <int D, bool FP8>
int64_t attention_tc_bytes(cudaError_t &e)
{
    int ctas = 0;
    e = attention_tc_ctas<D, FP8>(ctas);
    return e == cudaSuccess ? (int64_t)ctas * ((int64_t)sizeof(PartDesc) + 2 * (int64_t)TcCfg<D, FP8>::kPart * 4) : 0;
}

template <int D, bool FP8>
cudaError_t attention_tc(const AttnParams &p, cudaStream_t stream)
{
    using C = TcCfg<D, FP8>;
    int ctas = 0;
    cudaError_t e = attention_tc_ctas<D, FP8>(ctas);
    if (e == cudaSuccess)
        e = launch_pdl(attention_tc_kernel<D, FP8>, ctas, kTcThreads, C::kSmem, stream, p);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)(2 * (D / 32)));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_tc_kernel<D, FP8>, p, ctas);
}

template <int D>
int64_t workspace_tc(bool fp8, cudaError_t &e)
{
    return fp8 ? attention_tc_bytes<D, true>(e) : attention_tc_bytes<D, false>(e);
}

template <int D>
cudaError_t attention_tc_d(const AttnParams &p, bool fp8, cudaStream_t stream)
{
    return fp8 ? attention_tc<D, true>(p, stream) : attention_tc<D, false>(p, stream);
}

#define DSPARK_ATTN_TC_DECLARE(D)                                 \
    extern template int64_t workspace_tc<D>(bool, cudaError_t &); \
    extern template cudaError_t attention_tc_d<D>(const AttnParams &, bool, cudaStream_t);
#define DSPARK_ATTN_TC_DEFINE(D)                           \
    template int64_t workspace_tc<D>(bool, cudaError_t &); \
    template cudaError_t attention_tc_d<D>(const AttnParams &, bool, cudaStream_t);

}  // namespace attn
}  // namespace dspark
