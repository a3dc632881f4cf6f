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
// the places (its keys stay in shared memory where the slice fits), the
// histograms and counts are summed over distributed shared memory, the two
// lists go to the workspace, and after a cluster barrier the pairs are copied
// by all warps of the cluster, four rows in flight per warp.  NC is the
// smallest power of two that gives every SM two CTAs, at most 16, and at
// least 512 places per CTA: a serving batch has enough (request, head) pairs,
// a single long request does not.  Bound: the weights' and positions' read
// and write, and the rows that move; on small n the barriers between passes.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <mutex>

#include "ctx_kv_internal.h"
#include "draft_attn_internal.h"

namespace cg = cooperative_groups;

namespace dspark {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kKeysMax = 16384;  // keys of a slice kept in shared memory (64 KB)

struct Shared {
    unsigned hist[256];   // this CTA's histogram, read by the others
    unsigned warp_sum[kWarps];
    unsigned total;       // block scan
    unsigned counts[2];   // this CTA's {equal} then {holes, movers}, read by the others
    unsigned bin, above;  // the pass's result
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

// Exclusive prefix sum over the block; every thread also gets the total.
__device__ __forceinline__ unsigned block_scan(unsigned v, Shared &sh, unsigned &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d)
            x += y;
    }
    if (lane == 31)
        sh.warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
        unsigned s = lane < kWarps ? sh.warp_sum[lane] : 0u, z = s;
#pragma unroll
        for (int d = 1; d < kWarps; d <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, z, d);
            if (lane >= d)
                z += y;
        }
        if (lane < kWarps)
            sh.warp_sum[lane] = z - s;
        if (lane == kWarps - 1)
            sh.total = z;
    }
    __syncthreads();
    const unsigned base = sh.warp_sum[warp];
    total = sh.total;
    __syncthreads();
    return base + x - v;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictParams p, int cluster_size)
{
    pdl_enter();
    extern __shared__ uint32_t keys[];
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int NC = cluster_size;
    const int64_t bh = blockIdx.x / NC;
    const int b = (int)(bh / p.num_kv_heads), h = (int)(bh - (int64_t)b * p.num_kv_heads);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const int n = __ldg(p.context_lens + b);
    const bool bad = n < 0 || n > p.stride || n > p.table_blocks * p.block_size;
    const float *w = p.weights + bh * p.stride;
    const int32_t *pos = p.positions + bh * p.stride;
    float *wo = p.weights_out + bh * p.stride;
    int32_t *po = p.positions_out + bh * p.stride;
    const bool copies = wo != w, copies_pos = po != pos;
    const bool cut = !bad && n > p.budget;
    if (h == 0 && rank == 0 && tid == 0) {
        p.new_lens[b] = cut ? (int32_t)p.budget : n;
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
    if (!cut)
        return;  // the same for every CTA of the cluster
    const int budget = (int)p.budget;
    const int64_t first_recent = (int64_t)__ldg(p.seq_lens + b) - p.recent;
    const int per = (n + NC - 1) / NC;
    const int lo = min(n, rank * per), hi = min(n, lo + per);
    const bool in_smem = per <= kKeysMax;
    auto key_of = [&](int j) {
        const int at = pos[j];
        return sort_key(w[j], at < p.sinks || at >= first_recent);
    };
    if (in_smem)
        for (int j = lo + tid; j < hi; j += kThreads)
            keys[j - lo] = key_of(j);
    auto key = [&](int j) { return in_smem ? keys[j - lo] : key_of(j); };

    // ---- the budget-th largest key
    uint32_t prefix = 0;
    unsigned need = (unsigned)budget;  // still to take among the keys that agree with the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kThreads)
            sh.hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int j = lo + tid; j < hi; j += kThreads) {
            const uint32_t k = key(j);
            if ((k & mask) == prefix)
                atomicAdd(&sh.hist[(k >> shift) & 255u], 1u);
        }
        cluster.sync();
        // thread i < 256 sums bin 255 - i over the cluster; the scan then counts from the top
        unsigned v = 0;
        if (tid < 256)
            for (int c = 0; c < NC; c++)
                v += cluster.map_shared_rank(&sh, c)->hist[255 - tid];
        unsigned total;
        const unsigned before = block_scan(v, sh, total);
        if (tid < 256 && before < need && before + v >= need) {
            sh.bin = 255u - (unsigned)tid;
            sh.above = before;
        }
        cluster.sync();  // the result is there, and every CTA has read the histograms
        prefix |= sh.bin << shift;
        need -= sh.above;
    }
    // keys > prefix are kept, and the first `need` of those equal to it

    // ---- how many equal keys lie in the slices before this one
    const int chunk = (hi - lo + kThreads - 1) / kThreads;  // consecutive places per thread
    const int j0 = min(hi, lo + tid * chunk), j1 = min(hi, j0 + chunk);
    unsigned eq = 0;
    for (int j = j0; j < j1; j++)
        eq += key(j) == prefix;
    unsigned total;
    unsigned eq_before = block_scan(eq, sh, total);
    if (tid == 0)
        sh.counts[0] = total;
    cluster.sync();
    for (int c = 0; c < rank; c++)
        eq_before += cluster.map_shared_rank(&sh, c)->counts[0];
    cluster.sync();

    // ---- holes (given up, below budget) and movers (kept, at or above it)
    unsigned holes = 0, movers = 0, e = eq_before;
    for (int j = j0; j < j1; j++) {
        const uint32_t k = key(j);
        const bool keep = k > prefix || (k == prefix && e++ < need);
        holes += !keep && j < budget;
        movers += keep && j >= budget;
    }
    unsigned nh, nm;
    unsigned hole_at = block_scan(holes, sh, nh), mover_at = block_scan(movers, sh, nm);
    if (tid == 0)
        sh.counts[0] = nh, sh.counts[1] = nm;
    cluster.sync();
    unsigned moves = 0;
    for (int c = 0; c < NC; c++) {
        const Shared *o = cluster.map_shared_rank(&sh, c);
        if (c < rank)
            hole_at += o->counts[0], mover_at += o->counts[1];
        moves += o->counts[0];
    }
    int32_t *hole_list = p.lists + bh * 2 * p.list_len, *mover_list = hole_list + p.list_len;
    e = eq_before;
    for (int j = j0; j < j1; j++) {
        const uint32_t k = key(j);
        const bool keep = k > prefix || (k == prefix && e++ < need);
        if (j < budget) {
            if (!keep)
                hole_list[hole_at++] = j;
            else {
                if (copies)
                    wo[j] = w[j];
                if (copies_pos)
                    po[j] = pos[j];
            }
        } else if (keep) {
            mover_list[mover_at++] = j;
            if (copies)
                wo[j] = 0.0f;
            if (copies_pos)
                po[j] = -1;
        } else {
            wo[j] = 0.0f;
            po[j] = -1;
        }
    }
    cluster.sync();  // the lists are complete (and no CTA's shared memory is read any more)

    // ---- the moves
    const int warps = NC * kWarps, gw = rank * kWarps + warp;
    const int32_t *table = p.table + b * p.table_stride;
    const int clog = __ffs(p.row_bytes >> 4) - 1, chunks = 1 << clog;  // 16-byte words of a row: 8, 16, 32 or 64
    bool bad_block = false;
    auto row_of = [&](int j) -> unsigned char * {
        const int blk = j / p.block_size;
        const int64_t phys = __ldg(table + blk);
        if (phys < 0 || phys >= p.num_blocks) {
            bad_block = true;
            return nullptr;
        }
        return p.cache + ((phys * p.num_kv_heads + h) * p.block_size + (j - blk * p.block_size)) * (int64_t)p.row_bytes;
    };
    // each lane looks one pair up, then the warp copies the 32 rows
    for (unsigned base = gw * 32u; base < moves; base += warps * 32u) {
        const unsigned i = base + lane;
        unsigned char *from = nullptr, *to = nullptr;
        if (i < moves) {
            const int d = hole_list[i], s = mover_list[i];
            from = row_of(s), to = row_of(d);
            const float ws = w[s];
            const int32_t ps = pos[s];
            wo[d] = ws;
            po[d] = ps;
            if (!copies)
                wo[s] = 0.0f;
            if (!copies_pos)
                po[s] = -1;
            if (!to)
                from = nullptr;
        }
        const int count = (int)min(32u, moves - base);
        const int words = count * chunks;  // 16-byte words of these rows, lane-strided
        for (int x0 = 0; x0 < words; x0 += 32 * 4) {
            uint4 v[4];
            unsigned char *dst[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int x = x0 + k * 32 + lane;
                const int row = min(x >> clog, 31), c = x & (chunks - 1);
                const unsigned long long f = __shfl_sync(0xffffffffu, (unsigned long long)from, row);
                const unsigned long long t = __shfl_sync(0xffffffffu, (unsigned long long)to, row);
                dst[k] = nullptr;
                if (x < words && f != 0) {
                    v[k] = *reinterpret_cast<const uint4 *>(f + 16 * c);
                    dst[k] = reinterpret_cast<unsigned char *>(t + 16 * c);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (dst[k])
                    *reinterpret_cast<uint4 *>(dst[k]) = v[k];
        }
    }
    if (bad_block && p.error_flags)
        atomicOr(p.error_flags, kFlagBlockRange);
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
    static std::mutex mu;
    static bool attr_set[64];
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!attr_set[dev]) {
            e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysMax * 4);
            if (e != cudaSuccess)
                return e;
            attr_set[dev] = true;
        }
    }
    const int64_t pairs = (int64_t)p.num_requests * p.num_kv_heads;
    int nc = 1;
    while (nc < 16 && pairs * nc < 2 * sms && p.stride > 512 * nc)
        nc *= 2;
    const int64_t per = (p.stride + nc - 1) / nc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs * nc));
    cfg.blockDim = dim3((unsigned)kThreads);
    cfg.dynamicSmemBytes = (size_t)(per < kKeysMax ? per : kKeysMax) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)nc;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, evict_kernel, p, nc);
}

}  // namespace dspark
