// sm_103a kernel of the eviction of cached tokens by their accumulated
// attention weight.
//
// For each (request, KV head) the `budget` largest of n keys are kept.  A key
// is the weight as an unsigned number that grows with it (sign bit flipped,
// negative values complemented; NaN lowest, protected tokens above all), so
// the cut is the budget-th largest key, found by four passes over 8 bits from
// the top (a histogram of the keys that agree with the cut so far).  Keys
// above the cut are kept, of those equal to it the first in place order.
//
// Moving as little as possible: the kept tokens at places >= budget (movers)
// go to the places below budget that were given up (holes), the i-th to the
// i-th in place order.  There are equally many of both, sources lie at or
// above budget and destinations below, so no move reads what another writes
// and all run side by side; keeping the order instead would shift nearly
// every row behind the first hole.
//
// One cluster of NC CTAs per (request, KV head): each CTA ranks a slice of
// the places, its warps consecutive segments of it (ballots give the ranks in
// place order, whole lines are read and written), its keys in shared memory
// where the slice fits; the histograms and counts are summed over distributed
// shared memory, the two lists go to the workspace, and after a cluster
// barrier all threads move the pairs' weights and positions and turn the
// places into cache rows.  NC is the smallest power of two that gives every SM
// two CTAs, at most 16, and at least 512 places per CTA: a serving batch has
// enough (request, head) pairs, a single long request does not.
//
// The rows are copied by a second kernel, launched with programmatic overlap:
// it needs no cluster, so every SM takes part (in the first kernel two 131k
// contexts halved took 137 us: eight clusters of 16 CTAs do not spread over
// all SMs, nor do their registers allow 4 KB in flight per warp), and a warp
// needs nothing but the two lists.  Bound: the weights' and positions' read
// and write, and the rows that move (64 x 8 lists of 4,100 to 4,352 places cut to
// 4,096: 45 us, the bytes' time 15; two 131k contexts halved: 85 against 42); on
// small n the latency of the passes, some 3,500 cycles each.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <mutex>

#include "ctx_kv_internal.h"
#include "draft_attn_internal.h"

namespace cg = cooperative_groups;

namespace dspark {
namespace {

constexpr int kKeysMax = 16384;  // keys of a slice kept in shared memory (64 KB)

struct Shared {
    unsigned hist[256];        // this CTA's histogram, read by the others
    unsigned total[256];       // the cluster's
    unsigned warp_sum[32];
    unsigned counts[2];        // this CTA's {equal} then {holes, movers}, read by the others
    unsigned bin, above, same; // a pass's result: the cut's digit, keys above it, keys with it
};

__device__ __forceinline__ uint32_t sort_key(float w, bool keep_always)
{
    if (keep_always)
        return 0xffffffffu;
    if (w != w)
        return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);  // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;  // in [0x007fffff, 0xff800000]
}

// Sum over the warps before this one of their (warp-uniform) v, and over all.
template <int kWarps>
__device__ __forceinline__ unsigned warps_before(unsigned v, Shared &sh, unsigned &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0)
        sh.warp_sum[warp] = v;
    __syncthreads();
    const unsigned x = lane < kWarps ? sh.warp_sum[lane] : 0u;
    total = __reduce_add_sync(0xffffffffu, x);
    const unsigned before = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0u);
    __syncthreads();
    return before;
}

// Whether a length lies outside its bounds, and what the request keeps.
__device__ __forceinline__ bool bad_length(const EvictParams &p, int n)
{
    return n < 0 || n > p.stride || n > p.table_blocks * p.block_size;
}
__device__ __forceinline__ int32_t new_length(const EvictParams &p, int n)
{
    return !bad_length(p, n) && n > p.budget ? (int32_t)p.budget : n;
}

template <int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) evict_kernel(const EvictParams p, int NC)
{
    constexpr int kWarps = kThreads / 32;
    pdl_enter();
    extern __shared__ uint32_t keys[];
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int64_t bh = blockIdx.x / NC;
    const int b = (int)(bh / p.num_kv_heads), h = (int)(bh - (int64_t)b * p.num_kv_heads);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned below = (1u << lane) - 1u;  // the lanes before this one
    auto barrier = [&] {
        if (NC > 1)
            cluster.sync();
        else
            __syncthreads();
    };

    const int n = __ldg(p.context_lens + b);
    const bool bad = bad_length(p, n);
    const float *w = p.weights + bh * p.stride;
    const int32_t *pos = p.positions + bh * p.stride;
    float *wo = p.weights_out + bh * p.stride;
    int32_t *po = p.positions_out + bh * p.stride;
    const bool copies = wo != w, copies_pos = po != pos;
    const bool cut = !bad && n > p.budget;
    if (h == 0 && rank == 0 && tid == 0) {
        // The new lengths may take the place of the old ones (or of seq_lens),
        // which other CTAs of this grid still read: the second kernel writes
        // them, or, where there is none (no list can be too long), this one the
        // same numbers.
        if (p.list_len == 0)
            p.new_lens[b] = new_length(p, n);
        if (bad && p.error_flags)
            atomicOr(p.error_flags, kFlagLength);
    }
    // what no eviction touches: the whole row, or the places behind its length
    {
        const int64_t from = cut ? n : 0;
        for (int64_t j = from + rank * kThreads + tid; j < p.stride; j += (int64_t)NC * kThreads) {
            if (copies)
                wo[j] = w[j];
            if (copies_pos)
                po[j] = pos[j];
        }
    }
    if (!cut) {  // the same for every CTA of the cluster
        if (rank == 0 && tid == 0)
            p.counts[bh] = 0;
        return;
    }
    const int budget = (int)p.budget;
    const int64_t first_recent = (int64_t)__ldg(p.seq_lens + b) - p.recent;
    const int per = (n + NC - 1) / NC;
    const int lo = min(n, rank * per), hi = min(n, lo + per);
    const bool in_smem = per <= kKeysMax;
    // the warp's segment: whole groups of 32 places
    const int seg = ((per + kWarps - 1) / kWarps + 31) & ~31;
    const int s0 = min(hi, lo + warp * seg), s1 = min(hi, s0 + seg);
    for (int i = tid; i < 256; i += kThreads)
        sh.hist[i] = 0;
    __syncthreads();
    // ---- the keys, the first digit's histogram, and (not in place) the places
    // that no move will write: a hole is written again by its mover below
#pragma unroll 8
    for (int j = s0 + lane; j < s1; j += 32) {
        const float wv = w[j];
        const int32_t pv = pos[j];
        const uint32_t k = sort_key(wv, pv < p.sinks || pv >= first_recent);
        if (in_smem)
            keys[j - lo] = k;
        atomicAdd(&sh.hist[k >> 24], 1u);
        if (copies)
            wo[j] = j < budget ? wv : 0.0f;
        if (copies_pos)
            po[j] = j < budget ? pv : -1;
    }
    auto key = [&](int j) {
        if (in_smem)
            return keys[j - lo];
        const int32_t pv = pos[j];
        return sort_key(w[j], pv < p.sinks || pv >= first_recent);
    };

    // ---- the budget-th largest key
    uint32_t prefix = 0;
    unsigned need = (unsigned)budget;  // still to take among the keys that agree with the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (shift < 24) {
            for (int i = tid; i < 256; i += kThreads)
                sh.hist[i] = 0;
            __syncthreads();
            const uint32_t mask = 0xffffffffu << (shift + 8);
            for (int j = s0 + lane; j < s1; j += 32) {
                const uint32_t k = key(j);
                if ((k & mask) == prefix)
                    atomicAdd(&sh.hist[(k >> shift) & 255u], 1u);
            }
        }
        barrier();
        if (tid < 256) {  // one bin per thread: the cluster's loads go out together
            unsigned v = sh.hist[tid];
            if (NC > 1) {
                v = 0;
#pragma unroll 8
                for (int c = 0; c < NC; c++)
                    v += cluster.map_shared_rank(&sh, c)->hist[tid];
            }
            sh.total[tid] = v;
        }
        __syncthreads();
        // lane l of warp 0 takes bins 255 - 8 l ... 248 - 8 l: counts from the top
        if (warp == 0) {
            unsigned v[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                v[i] = sh.total[255 - 8 * lane - i];
                sum += v[i];
            }
            unsigned x = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d)
                    x += y;
            }
            unsigned before = x - sum;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                if (before < need && before + v[i] >= need) {
                    sh.bin = 255u - 8 * lane - i;
                    sh.above = before;
                    sh.same = v[i];
                }
                before += v[i];
            }
        }
        barrier();  // the result is there, and every CTA has read the histograms
        prefix |= sh.bin << shift;
        need -= sh.above;
    }
    // keys > prefix are kept, and the first `need` of the `same` equal to it
    const bool ties = need < sh.same;

    // ---- equal keys before this warp's segment, where only some of them are kept
    unsigned eq_before = 0;
    if (ties) {
        unsigned eq = 0, total;
        for (int j = s0 + lane; j - lane < s1; j += 32)
            eq += __popc(__ballot_sync(0xffffffffu, j < s1 && key(j) == prefix));
        eq_before = warps_before<kWarps>(eq, sh, total);
        if (tid == 0)
            sh.counts[0] = total;
        barrier();
        for (int c = 0; c < rank; c++)
            eq_before += cluster.map_shared_rank(&sh, c)->counts[0];
        barrier();
    }
    // whether place j (one per lane) stays; e: equal keys before the group of 32
    auto stays = [&](int j, unsigned &e) {
        const uint32_t k = j < s1 ? key(j) : 0u;
        bool keep = k >= prefix;
        if (ties) {
            const unsigned same = __ballot_sync(0xffffffffu, j < s1 && k == prefix);
            keep = k > prefix || (k == prefix && e + __popc(same & below) < need);
            e += __popc(same);
        }
        return keep && j < s1;
    };

    // ---- holes (given up, below budget) and movers (kept, at or above it)
    unsigned holes = 0, movers = 0, e = eq_before;
    for (int j = s0 + lane; j - lane < s1; j += 32) {
        const bool keep = stays(j, e);
        holes += __popc(__ballot_sync(0xffffffffu, j < s1 && !keep && j < budget));
        movers += __popc(__ballot_sync(0xffffffffu, keep && j >= budget));
    }
    unsigned nh, nm;
    unsigned hole_at = warps_before<kWarps>(holes, sh, nh), mover_at = warps_before<kWarps>(movers, sh, nm);
    if (tid == 0)
        sh.counts[0] = nh, sh.counts[1] = nm;
    barrier();
    unsigned moves = 0;
    for (int c = 0; c < NC; c++) {
        const Shared *o = NC > 1 ? cluster.map_shared_rank(&sh, c) : &sh;
        if (c < rank)
            hole_at += o->counts[0], mover_at += o->counts[1];
        moves += o->counts[0];
    }
    int32_t *hole_list = p.lists + bh * 2 * p.list_len, *mover_list = hole_list + p.list_len;
    e = eq_before;
    for (int j = s0 + lane; j - lane < s1; j += 32) {
        const bool keep = stays(j, e);
        const bool hole = j < s1 && !keep && j < budget, mover = keep && j >= budget;
        const unsigned hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
        if (hole)
            hole_list[hole_at + __popc(hb & below)] = j;
        if (mover)
            mover_list[mover_at + __popc(mb & below)] = j;
        hole_at += __popc(hb), mover_at += __popc(mb);
        if (j < s1 && j >= budget && !keep) {  // in place: given up beyond the budget
            if (!copies)
                wo[j] = 0.0f;
            if (!copies_pos)
                po[j] = -1;
        }
    }
    if (rank == 0 && tid == 0)
        p.counts[bh] = (int32_t)moves;
    barrier();  // the lists are complete (and no CTA's shared memory is read any more)

    // ---- the weights and positions move, a pair per thread; its places become rows of the cache
    const int32_t *table = p.table + b * p.table_stride;
    bool bad_block = false;
    auto row_of = [&](int j) -> uint32_t {
        const int blk = j / p.block_size;
        const int64_t phys = __ldg(table + blk);
        if (phys < 0 || phys >= p.num_blocks) {
            bad_block = true;
            return ~0u;
        }
        return (uint32_t)((phys * p.num_kv_heads + h) * p.block_size + (j - blk * p.block_size));
    };
#pragma unroll 2
    for (unsigned i = (unsigned)(rank * kThreads + tid); i < moves; i += (unsigned)(NC * kThreads)) {
        const int d = hole_list[i], s = mover_list[i];
        const float wv = w[s];
        const int32_t pv = pos[s];
        const uint32_t to = row_of(d), from = row_of(s);
        wo[d] = wv;
        po[d] = pv;
        if (!copies)
            wo[s] = 0.0f;
        if (!copies_pos)
            po[s] = -1;
        hole_list[i] = (int32_t)to;
        mover_list[i] = (int32_t)(to == ~0u ? ~0u : from);
    }
    if (bad_block && p.error_flags)
        atomicOr(p.error_flags, kFlagBlockRange);
}

// Copies the rows of the lists (blockIdx.x is the (request, KV head) pair,
// blockIdx.y its share of the moves) and writes the new lengths.
__global__ void __launch_bounds__(256, 3) move_kernel(const EvictParams p)
{
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.y == 0 && threadIdx.x == 0 && blockIdx.x % p.num_kv_heads == 0) {
        const int b = blockIdx.x / p.num_kv_heads;  // nobody else reads or writes its lengths any more
        p.new_lens[b] = new_length(p, __ldg(p.context_lens + b));
    }
    const unsigned moves = (unsigned)p.counts[blockIdx.x];
    const int32_t *holes = p.lists + (int64_t)blockIdx.x * 2 * p.list_len, *movers = holes + p.list_len;
    const int clog = __ffs(p.row_bytes >> 4) - 1, chunks = 1 << clog;  // 16-byte words of a row: 8, 16, 32 or 64
    const unsigned pairs = min(32u, 256u >> clog);                     // rows a warp copies at once: 8 words per lane
    const unsigned step = gridDim.y * 8u * pairs;
    // lane i < pairs holds the rows of pair base + i
    auto look = [&](unsigned base, uint32_t &from, uint32_t &to) {
        from = to = ~0u;
        if (lane < pairs && base + lane < moves)
            from = (uint32_t)movers[base + lane], to = (uint32_t)holes[base + lane];
    };
    uint32_t from, to;
    unsigned base = (blockIdx.y * 8u + warp) * pairs;
    look(base, from, to);
    for (; base < moves; base += step) {
        uint4 v[8];
        uint32_t next_from, next_to;
        look(base + step, next_from, next_to);
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int x = k * 32 + lane, row = x >> clog;
            const uint32_t f = __shfl_sync(0xffffffffu, from, row & 31);
            if (row < pairs && f != ~0u)
                v[k] = *reinterpret_cast<const uint4 *>(p.cache + (int64_t)f * p.row_bytes + 16 * (x & (chunks - 1)));
        }
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int x = k * 32 + lane, row = x >> clog;
            const uint32_t f = __shfl_sync(0xffffffffu, from, row & 31), t = __shfl_sync(0xffffffffu, to, row & 31);
            if (row < pairs && f != ~0u)
                *reinterpret_cast<uint4 *>(p.cache + (int64_t)t * p.row_bytes + 16 * (x & (chunks - 1))) = v[k];
        }
        from = next_from, to = next_to;
    }
}

}  // namespace

namespace {

template <int kThreads, int kBlocks>
cudaError_t launch(const EvictParams &p, int64_t pairs, int nc, int dev, cudaStream_t stream)
{
    static std::mutex mu;
    static bool attr_set[64];
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!attr_set[dev]) {
            cudaError_t e = cudaFuncSetAttribute(evict_kernel<kThreads, kBlocks>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(evict_kernel<kThreads, kBlocks>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysMax * 4);
            if (e != cudaSuccess)
                return e;
            attr_set[dev] = true;
        }
    }
    const int64_t per = (p.stride + nc - 1) / nc;
    const size_t smem = (size_t)(per < kKeysMax ? per : kKeysMax) * 4;
    return launch_pdl_grid(evict_kernel<kThreads, kBlocks>, dim3((unsigned)(pairs * nc)), kThreads, smem, nc, stream, p, nc);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictParams &p, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    const int64_t pairs = (int64_t)p.num_requests * p.num_kv_heads;
    int nc = 1;
    while (nc < 16 && pairs * nc < 2 * sms && p.stride > 512 * nc)
        nc *= 2;
    // pairs enough for every SM: 256 threads, so that all are there at once
    e = pairs * nc > sms ? launch<256, 4>(p, pairs, nc, dev, stream) : launch<512, 2>(p, pairs, nc, dev, stream);
    if (e != cudaSuccess || p.list_len == 0)
        return e;
    // the moves: three CTAs per SM over all pairs, none of them with less than
    // 8 rows a warp to copy where the lists are full
    const int64_t most = (p.list_len + 63) / 64;
    int64_t shares = (3 * (int64_t)sms + pairs - 1) / pairs;
    shares = shares < most ? shares : most;
    return launch_pdl_grid(move_kernel, dim3((unsigned)pairs, (unsigned)shares), 256, 0, 0, stream, p);
}

}  // namespace dspark
