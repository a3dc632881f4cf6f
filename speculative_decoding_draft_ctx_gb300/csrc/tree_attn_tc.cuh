// The drafted tokens' attention on the 5th-generation tensor cores, for
// requests of more than a few query rows (tcgen05 + tensor memory, sm_103a).
// Mathematics, rows, items, splitting and masking as in tree_attn_mma.cuh.
//
// Why.  With r rows of queries a cached token of D 128 brings 512 bytes and
// 512 r flops: the card's rates balance at r = 283, but mma.sync, whose
// operands pass through registers, is bound by issue from r = 56 on (64
// requests x 7 tokens x 8 heads: 234 us, this kernel 193, memory time 136; two
// trees of 64 over 131k tokens: 848 us, this kernel 248, its products' time 132).
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
//  - producer warps (2 for K, 2 for V): gather the tiles through the block
//    table into separate rings with 16-byte asynchronous copies, bf16 straight
//    into the operands' 128-byte swizzle, fp8 as codes that the warp turns into
//    fp16 in place, once per tile instead of once per row tile (a bulk copy per
//    row, 64 to 128 bytes, took 131 against 108 us on ragged fp8 trees);
//  - a warp per stream issues S = Q K^T (depth D) and O += P V (V as the cache
//    holds it: its N direction contiguous).  An MMA of 128 rows takes 64 cycles
//    for any width up to 128, so scores come 128 keys at a time (half tiles
//    with two buffers took the wait out of the softmax but doubled the first
//    product: 395 against 293 us on two 131k contexts), while the weights of
//    the first 64 keys go into the second product as soon as they are there.
//    With two row tiles the streams take turns with the scores' products:
//    interleaved, both streams' scores came late and both softmaxes ran at the
//    same time (298 against 271 us on two 131k contexts);
//  - softmax warps (8): 32 scores of a row at a time in registers, maximum,
//    base-2 exponentials with paired fp32 instructions, P back to tensor
//    memory.  The output is rescaled only when a row's weights would exceed
//    2^kMost otherwise: until then they exceed 1, which costs neither range nor
//    precision.  Over an fp8 cache fp16's range is used up by kLift but for one
//    octave.
//
// Loops are rolled where a role's straight-line code would not stay in the
// instruction caches beside the others' (unrolled, a warp's instruction took
// about ten cycles), and tiles without a mask have loops of their own.  14
// warps leave 128 registers a thread.  What bounds it now: with two row tiles
// the softmax (about 2,500 of 4,300 cycles a tile, where the same loops alone
// on an SM take 1,800), with one the tiles' arrival (a stage is held from its
// copy until its stream's softmax is done with the tile before).
// Every wait is bounded; on expiry the CTA raises DSPARK_FLAG_TIMEOUT, stops
// issuing, waits for its copies and products in flight, frees its tensor
// memory and returns.
#pragma once

#include "tc_ptx.cuh"
#include "tree_attn_mma.cuh"

namespace dspark {
namespace attn {

constexpr int kTcThreads = 448, kKeysTc = 128;  // 8 softmax warps, 4 producers, 2 that issue the products
constexpr int kProducers = 4, kItemCostTc = 6;   // EXTRA of Walk, in tiles of kKeysTc keys
// The largest weight 2^(s - m) that waits for a rescale, as an exponent: fp32
// sums and bf16 weights have room for any; fp16 weights begin at 2^kLift and
// end below 2^16 (a score is off by 2^-4 at most where kLift is taken off).
constexpr float kMost = 8.0f, kMostFp8 = kLift + 1.0f;

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <int D, bool FP8>
struct TcCfg {
    // Even: where the streams take turns, a stage belongs to one of them within
    // an item, so that neither is ever two phases off a stage's barrier.
    static constexpr int kStagesK = D == 64 ? 4 : 2, kStagesV = D == 64 ? 4 : 2;
    static constexpr int kTileBytes = kKeysTc * D * 2;    // one K or V tile, 16-bit
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kRow = 2 * D * (FP8 ? 1 : 2);    // bytes of a cached token
    static constexpr int kSmem = 1024 + 2 * kQBytes + (kStagesK + kStagesV) * kTileBytes;
    static constexpr int kRowPart = (D + 2) * 128;        // floats of one row tile's part
    static constexpr int kPart = 2 * kRowPart;
    static_assert(kSmem + 6 * 1024 <= 227 * 1024, "shared memory");
};

// 64-key halves of the n tiles at w: the second half of a request's last tile
// is left out where no token lies in it.
template <typename W>
__device__ __forceinline__ int tile_halves(const W &w, int n)
{
    return 2 * n - (w.finished() && w.rq.ctx + w.rq.nq <= (w.t1 - 1) * kKeysTc + kKeysTc / 2 ? 1 : 0);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kTcThreads, 1) attention_tc_kernel(const __grid_constant__ AttnParams p)
{
    using C = TcCfg<D, FP8>;
    using namespace tc;
    constexpr int NK = C::kStagesK, NV = C::kStagesV;
    // tensor-memory columns: scores of stream s at 128 s, output at 256 + 128 s
    constexpr uint32_t kO[2] = {256, 256 + 128};
    constexpr uint32_t kIdQK = idesc(FP8, false, 128, kKeysTc), kIdPV = idesc(FP8, true, 128, D);
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (tc::saddr(smem_raw) & 1023u)) & 1023u);
    unsigned char *sq = smem, *sk = smem + 2 * C::kQBytes, *sv = sk + NK * C::kTileBytes;
    __shared__ uint64_t kfull[NK], kempty[NK], vfull[NV], vempty[NV], qfull[2], sfull[2], pfull[4], ofull[2], jfull, jempty, go1, done[2];
    __shared__ uint32_t tmem_slot, live[8][4];
    __shared__ uint32_t rows[kProducers][2][64];  // cache rows of each producer's tile and its next; ~0: not there
    __shared__ int abort_flag, lock;
    __shared__ int bad[16];  // item number + 1 where infinities or NaN came up among an item's drafted V
    __shared__ float join_ml[256];
    __shared__ int64_t scratch[kTcThreads / 32 + 4];
    const Patience limit{&abort_flag, p.wait_ns};

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < NK; s++) {
            bar_init(kfull + s, 64 + 2);  // two producer warps' copies, and their live masks
            bar_init(kempty + s, 2);  // both streams
        }
        for (int s = 0; s < NV; s++) {
            bar_init(vfull + s, 64);
            bar_init(vempty + s, 2);
        }
        for (int s = 0; s < 2; s++) {
            bar_init(qfull + s, 128);
            bar_init(ofull + s, 1);
            bar_init(sfull + s, 1);
            bar_init(pfull + 2 * s, 4);
            bar_init(pfull + 2 * s + 1, 4);
            bar_init(done + s, 1);
        }
        bar_init(&jfull, 128);
        bar_init(&jempty, 128);
        bar_init(&go1, 8);
        abort_flag = 0, lock = 0;
        for (int i = 0; i < 16; i++)
            bad[i] = 0;
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
    using W = Walk<256, kKeysTc, kItemCostTc>;
    const Find f = find_request<kTcThreads>(p.num_requests, scratch,
                                            [&](int b) { return W::units(p, request(p, b, mask_limit, flags)); });
    const Shares shares(f.total, ctas);
    PartDesc *descs = reinterpret_cast<PartDesc *>(p.parts);
    float *parts = p.parts + (int64_t)ctas * (sizeof(PartDesc) / 4);
    if (tid == 0)
        descs[cta].last = -1, descs[cta].bad[0] = 0, descs[cta].bad[1] = 0;
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;
    // every role walks the CTA's share on its own, item by item
    W w;
    w.start(p, f.b >= 0 ? shares.start(cta) : 0, f.b >= 0 ? shares.start(cta + 1) : 0, f.b, f.before, mask_limit);

    if (warp >= 12) {
        // ------------------------------------------------------------ the issuing warps, one per stream
        // The whole warp walks and waits, one lane issues: in a branch of one
        // lane the descriptors went through vector registers and an MMA took
        // 106 cycles to issue, of any size.
        const bool leader = elect();
        auto stream = [&](auto sc) {
            constexpr int s = decltype(sc)::value;
            int base = 0;                // tiles consumed before this item
            int nq0 = 0, nq1 = 0, ngo = 0;  // uses of qfull[0], qfull[1] and go1
            uint32_t par = 0;            // parities of the stream's two pfull
            bool ok = true;
            while (w.more() && ok) {
                const int n = w.t1 - w.t0;
                const bool two = w.rq.nq * p.group - w.row0() > 128;
                const int halves = tile_halves(w, n);
                const int steps = two ? n : s == 0 ? (n + 1) >> 1 : n >> 1;
                auto tile_of = [&](int k) { return two ? k : 2 * k + s; };
                auto wait = [&](uint64_t *bar, uint32_t parity) {
                    ok = ok && bar_wait(bar, parity, limit);
                    ok = __all_sync(0xffffffffu, ok);
                };
                // a stage is free when both streams are done with it; where the
                // streams take turns, the other one's word is given with this one's
                auto release = [&](uint64_t *bar) {
                    mma_commit(bar);
                    if (!two)
                        bar_arrive(bar);
                };
                auto qk = [&](int k) {
                    const int st = (base + tile_of(k)) % NK;
                    fence_async();
                    fence_after();
                    if (leader) {
                        pick<NK>(st, [&](auto stc) {
                            constexpr int S = decltype(stc)::value;
                            const uint32_t b = tc::saddr(sk) + S * C::kTileBytes;
                            auto issue = [&](uint32_t a) {
#pragma unroll
                                for (int k = 0; k < D / 16; k++)
                                    mma_ss(tmem + 128 * s, desc128(a + (k / 4) * 16384 + (k % 4) * 32, 16),
                                           desc128(b + (k / 4) * 16384 + (k % 4) * 32, 16), kIdQK, k != 0);
                            };
                            if (s == 1 && two)
                                issue(tc::saddr(sq) + C::kQBytes);
                            else
                                issue(tc::saddr(sq));
                            mma_commit(sfull + s);
                            release(kempty + S);
                        });
                    }
                    __syncwarp();
                };
                auto pv = [&](int k, int h, bool last) {
                    const int st = (base + tile_of(k)) % NV;
                    fence_async();
                    fence_after();
                    if (leader) {
                        pick<NV>(st, [&](auto stc) {
                            pick<2>(h, [&](auto hc) {
                                constexpr int S = decltype(stc)::value, H = decltype(hc)::value;
                                const uint32_t b = tc::saddr(sv) + S * C::kTileBytes + H * 8192;  // 64 keys of 128 bytes
#pragma unroll
                                for (int i = 0; i < 4; i++)
                                    mma_ts(tmem + kO[s], tmem + 128 * s + 32 * H + 8 * i, desc128(b + i * 2048, 16384), kIdPV,
                                           i != 0 || H != 0 || k != 0);
                                if (last)
                                    release(vempty + S);
                            });
                        });
                    }
                    __syncwarp();
                };
                // One stream's products at a time: interleaved, both streams' scores
                // came late and their softmax ran at the same time.
                auto take = [&]() {
                    if (leader && two) {
                        const unsigned long long t0 = gtimer();
                        while (atomicExch(&lock, 1) != 0 && !*limit.abort)
                            if (gtimer() - t0 > limit.ns)
                                *limit.abort = 1;
                    }
                    __syncwarp();
                };
                auto give = [&]() {
                    if (leader && two)
                        atomicExch(&lock, 0);
                    __syncwarp();
                };
                auto kwait = [&](int k) {
                    const int x = base + tile_of(k);
                    wait(kfull + x % NK, (uint32_t)(x / NK) & 1u);
                };
                // Where the streams share the rows, stream 1 waits for both
                // streams' softmax to be here first.  Over items of two row tiles
                // the streams drift apart by as many items as tiles fit the ring;
                // with both here everything before this item is done, and the
                // phases below are the next ones of their barriers.
                if (steps > 0) {
                    if (s == 1 && !two)
                        wait(&go1, (uint32_t)(ngo++) & 1u);
                    wait(qfull + (two ? s : 0), (uint32_t)(two && s == 1 ? nq1 : nq0) & 1u);
                }
                nq0++;
                nq1 += two;
                if (steps > 0 && ok) {
                    kwait(0);
                    if (ok)
                        qk(0);
                }
#pragma unroll 1
                for (int k = 0; k < steps && ok; k++) {
                    const int x = base + tile_of(k);
                    const bool both = 2 * tile_of(k) + 1 != halves;
                    wait(vfull + x % NV, (uint32_t)(x / NV) & 1u);
                    if (k + 1 < steps)
                        kwait(k + 1);
                    wait(pfull + 2 * s, par & 1u);
                    par ^= 1u;
                    if (ok)
                        pv(k, 0, !both);
                    if (both && ok) {
                        wait(pfull + 2 * s + 1, (par >> 1) & 1u);
                        par ^= 2u;
                    }
                    if (both && ok)
                        pv(k, 1, true);
                    take();
                    if (k + 1 < steps && ok)
                        qk(k + 1);
                    give();
                }
                if (steps > 0 && leader)
                    mma_commit(ofull + s);
                __syncwarp();
                base += n;
                w.next(p);
            }
            if (leader)
                mma_commit(done + s);
            __syncwarp();
        };
        if (warp == 12)
            stream(std::integral_constant<int, 0>{});
        else
            stream(std::integral_constant<int, 1>{});
    } else if (warp >= 8) {
        // ------------------------------------------------------------ producers
        // Two warps copy K, two V, each 64 rows of every tile.  While a warp
        // copies a tile it has the next one's rows fetched into L2, so that what
        // is in flight is not bounded by the rings, and looks up the blocks of
        // the one after.  bf16 lands in place and the copies themselves arrive
        // on the tile's barrier; fp8 lands as codes, is converted, and the next
        // tile is issued before that where its stage is free already.
        const int pw = warp - 8, half = pw >> 1, sub = pw & 1;  // half 0: K, 1: V
        const bool is_v = half != 0;
        const unsigned char *cache = p.cache + half * (C::kRow / 2);
        unsigned char *ring = is_v ? sv : sk;
        uint64_t *fulls = is_v ? vfull : kfull, *empties = is_v ? vempty : kempty;
        const int ns = is_v ? NV : NK;
        int phys[2], off[2];  // of the tile looked up last: rows lane and lane + 32 of the warp's; off < 0: past the end
        int look_tile = w.t0, look_head = 0, looked = 0;  // looked: tiles looked up, two ahead while there are any
        W lw = w;  // the walk of the look-ups; w is the walk of the tiles that are finished
        auto look = [&]() {
            off[0] = off[1] = -1;
            if (!lw.more())
                return;
            looked++;
            const int len = lw.rq.ctx + lw.rq.nq;
            look_head = lw.head();
#pragma unroll
            for (int g = 0; g < 2; g++) {
                const int j = look_tile * kKeysTc + 64 * sub + 32 * g + lane, blk = block_of(p, j);
                phys[g] = 0;
                if (j < len) {
                    off[g] = j - blk * p.block_size;
                    phys[g] = __ldg(p.table + lw.b * p.table_stride + blk);
                }
            }
            if (++look_tile >= lw.t1) {
                lw.next(p);
                look_tile = lw.t0;
            }
        };
        // the rows' numbers, once the block numbers have come, and the rows into L2
        auto resolve = [&](int slot) {
#pragma unroll
            for (int g = 0; g < 2; g++) {
                uint32_t at = ~0u;
                if (off[g] >= 0) {
                    if (phys[g] < 0 || phys[g] >= p.num_blocks) {
                        flags |= kFlagBlockRange;
                    } else {
                        at = (uint32_t)(((int64_t)phys[g] * p.num_kv_heads + look_head) * p.block_size + off[g]);
                        const unsigned char *row = cache + (int64_t)at * C::kRow;
#pragma unroll
                        for (int y = 0; y < C::kRow / 2; y += 128)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(row + y));
                    }
                }
                rows[pw][slot][32 * g + lane] = at;
            }
            __syncwarp();
        };
        constexpr int kW = D * (FP8 ? 1 : 2) / 16, kR = 32 / kW;  // 16-byte words of a row's half; rows a warp takes at once
        constexpr int kB = 64 / kR < 8 ? 64 / kR : 8;
        const int c = lane % kW, r = lane / kW;
        bool ok = true;
        // issues the copies of tile number x of the share (its rows are resolved),
        // and resolves the next one's
        auto issue = [&](int x) {
            const uint32_t dst0 = tc::saddr(ring) + (x % ns) * C::kTileBytes;
            const uint32_t *from = rows[pw][x & 1];
            resolve((x & 1) ^ 1);
            look();
#pragma unroll 1
            for (int y0 = 0; y0 < 64; y0 += kR * kB) {
                uint32_t src[kB];
#pragma unroll
                for (int i = 0; i < kB; i++)
                    src[i] = from[y0 + i * kR + r];
#pragma unroll
                for (int i = 0; i < kB; i++) {
                    const int y = 64 * sub + y0 + i * kR + r;
                    const uint32_t at = FP8 ? raw_at<D>(dst0, y, c) : dst0 + (c >> 3) * 16384 + y * 128 + (((c & 7) ^ (y & 7)) << 4);
                    cp16(at, src[i] != ~0u ? cache + (int64_t)src[i] * C::kRow + 16 * c : p.cache, src[i] != ~0u);
                }
            }
            if (!is_v) {
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    const unsigned bits = __ballot_sync(0xffffffffu, from[32 * g + lane] != ~0u);
                    if (lane == 0)
                        live[x & 7][2 * sub + g] = bits;
                }
            }
            if (FP8)
                cp_commit();
            __syncwarp();  // every lane is done with this tile's row numbers
        };
        auto free_parity = [&](int x) { return ((uint32_t)(x / ns) & 1u) ^ 1u; };
        int x = 0, item = 0, tile = w.t0, issued = 0;  // tile and item number of the share; the request's tile
        look();
        resolve(0);
        look();
        if (p.test_hold)
            looked = 0;  // test hook: nothing is copied, the other roles' waits run out
        for (; x < looked && ok; x++) {
            const int st = x % ns, key0 = tile * kKeysTc + 64 * sub;
            const bool drafted = is_v && key0 + 64 > w.rq.ctx;
            if (issued == x) {
                ok = bar_wait(empties + st, free_parity(x), limit);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                issue(x);
                issued++;
            }
            if (FP8 && x + 1 < looked && __all_sync(0xffffffffu, bar_test(empties + (x + 1) % ns, free_parity(x + 1)))) {
                issue(x + 1);
                issued++;
            }
            if constexpr (FP8) {
                if (issued > x + 1)  // the next tile's copies are in flight as well
                    cp_wait<1>();
                else
                    cp_wait<0>();
                __syncwarp();
                if (convert_rows<D, 64>(tc::saddr(ring) + st * C::kTileBytes, 64 * sub, drafted ? w.rq.ctx - tile * kKeysTc : kKeysTc))
                    bad[item & 15] = item + 1;
                fence_async();
            } else if (drafted) {
                // infinities and NaN among the drafted V: zeroed here, accounted for at the end
                asm volatile("cp.async.wait_all;" ::: "memory");
                unsigned char *dst = ring + st * C::kTileBytes;
#pragma unroll 1
                for (int y = 64 * sub + r; y < 64 * sub + 64; y += kR) {
                    if (tile * kKeysTc + y < w.rq.ctx)
                        continue;
                    uint4 *at = reinterpret_cast<uint4 *>(dst + (c >> 3) * 16384 + y * 128 + (((c & 7) ^ (y & 7)) << 4));
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
                        bad[item & 15] = item + 1;
                    }
                }
                fence_async();
            }
            if (!is_v && lane == 0)
                bar_arrive(fulls + st);  // the live masks
            if (FP8 || drafted)
                bar_arrive(fulls + st);
            else
                bar_arrive_copies(fulls + st);
            if (++tile >= w.t1) {
                w.next(p);
                tile = w.t0;
                item++;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ------------------------------------------------------------ softmax: a thread per query row
        const int s = warp >> 2, q4 = warp & 3, r = q4 * 32 + lane;
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const float ks = FP8 && p.k_scale ? __ldg(p.k_scale) : 1.0f, vs = FP8 && p.v_scale ? __ldg(p.v_scale) : 1.0f;
        const float base_scale = p.scale * kLog2e * ks;
        int base = 0, item_no = 0;
        int nS = 0, nO = 0;  // S tiles read, items whose output is done (of this stream)
        int nJ = 0;          // items whose rows the streams shared
        bool ok = true;
        while (w.more() && ok) {
            const int n = w.t1 - w.t0, rows = w.rq.nq * p.group;
            const int h = w.head(), row0 = w.row0();
            const bool two = rows - row0 > 128;
            const bool begun = w.begun(), finished = w.finished();
            const int rt = two ? s : 0, my = row0 + rt * 128 + r;
            const bool mine = my < rows, warp_live = row0 + rt * 128 + q4 * 32 < rows;
            const int i = mine ? my / p.group : 0, hq = h * p.group + (mine ? my - i * p.group : 0);
            const int halves = tile_halves(w, n);
            const int steps = two ? n : s == 0 ? (n + 1) / 2 : n / 2;  // tiles of the stream
            if (!two && n > 1 && lane == 0)
                bar_arrive(&go1);
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
#pragma unroll 4
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
#pragma unroll (FP8 ? 4 : 8)
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
            // Not 0, or a masked score's -inf would become NaN: 1 where the queries
            // are zeroed, else the least number where the product underflows (a
            // tiny scale times the power of two of a tiny query over fp8).
            c = c == 0.0f ? (base_scale == 0.0f ? 1.0f : 1.4e-45f) : fabsf(c);
            const uint64_t c2 = pr(c, c);
            float m = -INFINITY, l = 0.0f;  // what the row subtracts (scaled, base 2), the sum of weights

            for (int k = 0; k < steps; k++) {
                const int j = two ? k : 2 * k + s;
                const int key0 = (w.t0 + j) * kKeysTc;
                const int nh = 2 * j + 1 == halves ? 1 : 2;  // 64-key halves that hold tokens
                const uint32_t ts = tmem + lanes + 128 * s;
                ok = ok && bar_wait(sfull + s, (uint32_t)nS & 1u, limit);
                nS++;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                fence_after();
                if (warp_live) {
                    const int lx = (base + j) & 7;
                    const bool masked = key0 + kKeysTc > w.rq.ctx || (live[lx][0] & live[lx][1] & live[lx][2] & live[lx][3]) != 0xffffffffu;
                    // bit b of visible(g): key key0 + 32 g + b is seen
                    auto visible = [&](int g) {
                        uint32_t vis = mine ? live[lx][g] : 0u;
                        const int a0 = key0 + 32 * g - w.rq.ctx;  // the drafted token of bit 0; below 0: context
                        if (a0 > -32) {
                            const int sh = a0 < 0 ? -a0 : 0, a = a0 < 0 ? 0 : a0;  // bits below sh are context
                            uint32_t t = 0xffffffffu;
                            if (p.mask_kind == 2) {
                                const uint64_t *words = p.tree_mask + (int64_t)(w.rq.q0 + i) * p.mask_words;
                                const int wd = a >> 6, bt = a & 63;
                                uint64_t y = wd < p.mask_words ? __ldg(words + wd) >> bt : 0ull;
                                if (bt > 32 && wd + 1 < p.mask_words)
                                    y |= __ldg(words + wd + 1) << (64 - bt);
                                t = (uint32_t)y;
                            }
                            const int room = (p.mask_kind == 1 ? min(w.rq.nq, i + 1) : w.rq.nq) - a;
                            t = room <= 0 ? 0u : room < 32 ? t & ((1u << room) - 1u) : t;
                            vis &= sh ? (t << sh) | ((1u << sh) - 1u) : t;
                        }
                        return vis;
                    };
                    // 32 scores, -inf where not seen
                    auto load32 = [&](auto gc, int g, uint32_t (&x)[32]) {
                        tmem_ld32(ts + 32 * g, x);
                        if constexpr (decltype(gc)::value) {
                            const uint32_t vis = masked ? visible(g) : 0xffffffffu;
#pragma unroll
                            for (int e = 0; e < 32; e++)
                                if (!((vis >> e) & 1u))
                                    x[e] = 0xff800000u;
                        }
                    };
                    // ---- maximum (the scores are read again below)
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    auto maxima = [&](auto gc) {
#pragma unroll 1
                        for (int g = 0; g < 2 * nh; g++) {
                            uint32_t x[32];
                            load32(gc, g, x);
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
#pragma unroll
                                for (int k2 = 0; k2 < 4; k2++)
                                    top[k2] = max3(top[k2], __uint_as_float(x[e + 2 * k2]), __uint_as_float(x[e + 2 * k2 + 1]));
                        }
                    };
                    if (__builtin_expect(masked, 0))
                        maxima(std::true_type{});
                    else
                        maxima(std::false_type{});
                    const float t = max3(fmaxf(top[0], top[1]), top[2], top[3]) * c;
                    const float most = !FP8 ? kMost : fabsf(t) < kLiftBelow ? kMostFp8 : 1.0f;
                    const bool grow = t > m + most || (m == -INFINITY && t > m);
                    if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
                        const float old = m;
                        m = fmaxf(m, reference_of<FP8>(t));
                        const float fr = old == m ? 1.0f : ex2(old - m);  // 0 from -inf
                        l *= fr;
                        if (k > 0) {
                            // the products so far are in: S of this tile came after them
#pragma unroll 1
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
                    // s c - m in one rounding shows m's own where that is large
                    // (scores beyond 2^24): the product is rounded first there
                    const bool apart = __any_sync(0xffffffffu, fabsf(mu) > 16777216.0f);
                    uint64_t sum0 = 0, sum1 = 0;
                    auto raise = [&](auto gc) {
#pragma unroll 1
                        for (int g = 0; g < 2 * nh; g++) {
                            uint32_t x[32], pk[16];
                            load32(gc, g, x);
                            if (decltype(gc)::value && apart) {
#pragma unroll
                                for (int e = 0; e < 32; e++)
                                    x[e] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(x[e]), c), mu));
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    float a0, a1;
                                    unpr(fma2(pr(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2, m2), a0, a1);
                                    x[e] = __float_as_uint(a0), x[e + 1] = __float_as_uint(a1);
                                }
                            }
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float a0 = ex2(__uint_as_float(x[e])), a1 = ex2(__uint_as_float(x[e + 1]));
                                const float a2 = ex2(__uint_as_float(x[e + 2])), a3 = ex2(__uint_as_float(x[e + 3]));
                                sum0 = add2(sum0, pr(a0, a1));
                                sum1 = add2(sum1, pr(a2, a3));
                                pk[e / 2] = pack2<FP8>(a0, a1);
                                pk[e / 2 + 1] = pack2<FP8>(a2, a3);
                            }
                            // columns 16 g .. of P lie over scores that are used up
                            tmem_st16(ts + 16 * g, pk);
                            if (g & 1) {  // a half's weights are out: its product may begin
                                tmem_wait_st();
                                fence_before();
                                __syncwarp();
                                if (lane == 0)
                                    bar_arrive(pfull + 2 * s + (g >> 1));
                            }
                        }
                    };
                    // Tiles without a mask run a short loop of their own: the
                    // instructions a warp has to fetch per tile are what bounds it.
                    if (__builtin_expect(masked || apart, 0))
                        raise(std::true_type{});
                    else
                        raise(std::false_type{});
                    float a0, a1;
                    unpr(add2(sum0, sum1), a0, a1);
                    l += a0 + a1;
                } else {
                    fence_before();
                    if (lane < nh)
                        bar_arrive(pfull + 2 * s + lane);
                    __syncwarp();
                }
            }
            if (!ok)
                break;
            // ---- the item ends here, or the CTA's share of it does
            if (steps > 0) {
                ok = bar_wait(ofull + s, (uint32_t)nO & 1u, limit);
                ok = __all_sync(0xffffffffu, ok);
                nO++;
            }
            fence_after();
            float y0 = 1.0f, y1 = 0.0f;  // factors of the two streams' sums
            if (!two) {
                if (s == 1) {
                    join_ml[r] = m, join_ml[128 + r] = l;
                    fence_before();
                    bar_arrive(&jfull);
                    // its output and statistics stay until stream 0 has read them
                    ok = ok && bar_wait(&jempty, (uint32_t)nJ & 1u, limit);
                } else {
                    ok = ok && bar_wait(&jfull, (uint32_t)nJ & 1u, limit);
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
            const bool is_bad = bad[item_no & 15] == item_no + 1;
            if ((two || s == 0) && warp_live) {
                const bool other = !two && n > 1;
                float *part = parts + ((int64_t)cta * 2 + (begun ? 1 : 0)) * C::kPart + rt * C::kRowPart + r;
                const bool direct = begun && finished;
                const float inv = l > 0.0f ? vs / l : l == 0.0f ? 0.0f : l;
                const int64_t at = (int64_t)(w.rq.q0 + i) * p.num_heads + hq;
                uint16_t *dst = p.out + at * D;
                // results go through this warp's own rows of the Q tile, which no
                // product reads any more, so that rows are written whole
                auto stage = [&](int y, int word) {
                    return reinterpret_cast<uint4 *>(sq + rt * C::kQBytes + (word >> 3) * 16384 + (q4 * 32 + y) * 128 + (((word & 7) ^ (y & 7)) << 4));
                };
#pragma unroll 1
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
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *stage(lane, (d + e) / 8) =
                                make_uint4(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]), pack_bf16x2(v[e + 4], v[e + 5]),
                                           pack_bf16x2(v[e + 6], v[e + 7]));
                    }
                }
                if (direct) {
                    __syncwarp();
                    constexpr int kOW = D / 8, kOR = 32 / kOW;  // 16-byte words of a row, rows at once
                    const int oc = lane % kOW;
#pragma unroll 1
                    for (int y = lane / kOW; y < 32; y += kOR) {
                        const int my2 = row0 + rt * 128 + q4 * 32 + y;
                        if (my2 >= rows)
                            break;
                        const int i2 = my2 / p.group;
                        *reinterpret_cast<uint4 *>(p.out + ((int64_t)(w.rq.q0 + i2) * p.num_heads + h * p.group + (my2 - i2 * p.group)) * D + 8 * oc) =
                            *stage(y, oc);
                    }
                    __syncwarp();
                }
                if (!direct)
                    part[D * 128] = m, part[(D + 1) * 128] = l;
                else if (mine) {
                    if (is_bad)
                        add_nonfinite<D, FP8>(p, w.b, w.rq, h, i, dst, 0, D);
                    p.lse[at] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
                }
            }
            fence_before();
            if (!two && s == 0)
                bar_arrive(&jempty);
            if (tid == 0) {
                if (begun && !finished) {
                    PartDesc &d = descs[cta];
                    d.q0 = w.rq.q0, d.rows = rows, d.row0 = row0, d.h = h, d.nq = w.rq.nq, d.ctx = w.rq.ctx, d.b = w.b;
                    d.last = w.last_cta(shares);
                }
                if (is_bad && !(begun && finished))
                    descs[cta].bad[begun ? 1 : 0] = 1;
            }
            base += n;
            item_no++;
            w.next(p);
        }
    }
    __syncthreads();
    if (warp == 12) {
        // every product has completed before the tensor memory is freed
        if (lane == 0) {
            const unsigned long long t0 = gtimer();
            for (int s = 0; s < 2; s++)
                while (!bar_try(done + s, 0) && !(flags & kFlagTimeout))
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

constexpr int kJoinDims = 16;

// Joins the parts of the item that CTA blockIdx.x began and did not finish:
// block y takes kJoinDims dims of row tile y / (D / kJoinDims), a thread per
// row.  Loads of several parts go out at a time: one after the other, an item
// over 19 CTAs took 30 us to join.
template <int D, bool FP8>
__global__ void __launch_bounds__(128) join_tc_kernel(const __grid_constant__ AttnParams p, int ctas)
{
    using C = TcCfg<D, FP8>;
    pdl_enter();
    const int r = threadIdx.x, rt = blockIdx.y / (D / kJoinDims), d0 = (blockIdx.y % (D / kJoinDims)) * kJoinDims;
    const PartDesc *descs = reinterpret_cast<const PartDesc *>(p.parts);
    const PartDesc d = descs[blockIdx.x];
    const int my = d.row0 + rt * 128 + r;
    if (d.last < 0 || my >= d.rows)
        return;
    const float *parts = p.parts + (int64_t)ctas * (sizeof(PartDesc) / 4);
    auto part = [&](int c) {
        return parts + ((int64_t)c * 2 + (c == (int)blockIdx.x ? 1 : 0)) * C::kPart + rt * C::kRowPart + r;
    };
    const int first = blockIdx.x;
    float m = -INFINITY;
    bool bad = false;
    for (int c0 = first; c0 <= d.last; c0 += 8) {  // the loads of eight parts at a time
        float v[8];
        int any[8];
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int c = min(c0 + k, d.last);
            v[k] = part(c)[D * 128], any[k] = descs[c].bad[c == first ? 1 : 0];
        }
#pragma unroll
        for (int k = 0; k < 8; k++)
            m = fmaxf(m, v[k]), bad |= any[k] != 0;
    }
    const float u = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, o[kJoinDims];
#pragma unroll
    for (int e = 0; e < kJoinDims; e++)
        o[e] = 0.0f;
    for (int c0 = first; c0 <= d.last; c0 += 4) {
        float v[4][kJoinDims], pm[4], pl[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const bool there = c0 + k <= d.last;
            const float *at = part(there ? c0 + k : d.last);
            pm[k] = there ? at[D * 128] : -INFINITY, pl[k] = there ? at[(D + 1) * 128] : 0.0f;
#pragma unroll
            for (int e = 0; e < kJoinDims; e++)
                v[k][e] = there ? at[(d0 + e) * 128] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float x = ex2(pm[k] - u);
            l = fmaf(pl[k], x, l);
#pragma unroll
            for (int e = 0; e < kJoinDims; e++)
                o[e] = fmaf(v[k][e], x, o[e]);
        }
    }
    const float vs = FP8 && p.v_scale ? __ldg(p.v_scale) : 1.0f;
    const float inv = l > 0.0f ? vs / l : l == 0.0f ? 0.0f : l;
    const int i = my / p.group, hq = d.h * p.group + (my - i * p.group);
    const int64_t at = (int64_t)(d.q0 + i) * p.num_heads + hq;
    if (d0 == 0)
        p.lse[at] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
#pragma unroll
    for (int e = 0; e < kJoinDims; e++)
        o[e] *= inv;
#pragma unroll
    for (int e = 0; e < kJoinDims; e += 8)
        *reinterpret_cast<uint4 *>(p.out + at * D + d0 + e) =
            make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]), pack_bf16x2(o[e + 4], o[e + 5]),
                       pack_bf16x2(o[e + 6], o[e + 7]));
    if (bad)
        add_nonfinite<D, FP8>(p, d.b, Request{d.q0, d.nq, d.ctx}, d.h, i, p.out + at * D, d0, d0 + kJoinDims);
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
            e = cudaFuncSetAttribute(attention_tc_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     TcCfg<D, FP8>::kSmem);
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
    return launch_pdl_grid(join_tc_kernel<D, FP8>, dim3((unsigned)ctas, (unsigned)(2 * (D / kJoinDims))), 128, 0, 0, stream, p, ctas);
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
