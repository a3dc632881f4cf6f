// New tokens' K and V into a page-scaled cache (sm_103a).
//
// Mathematics.  For a page and head, K and V apart: e = the least with max |x| <=
// 448 * 2^e over the finite new x, kept to [-32, 31] and to the page's scale where
// it holds context tokens; codes are e4m3(x * 2^-e).  448 = 1.75 * 2^8, so for
// max |x| = 1.f * 2^E, e = E - 8, or E - 7 where 1.f > 1.75.  x * 2^-e is exact
// in fp32, the code's rounding the only one.  A page whose scale grows has its
// codes divided by a power of two (page_scale.cuh).
//
// Work.  A unit is one (request, page, head); its tokens are read once: a
// thread keeps up to kHold 16-byte words while the CTA finds the maximum.  Lengths
// are on the device, so each CTA sums the requests' units itself and takes an
// equal share of them, as the attention does.  A CTA has 128 threads, so that
// a draft step's units (7 tokens of 512 bytes) are there all at once.
#include "draft_step_internal.h"
#include "page_scale.cuh"
#include "tree_attn_mma.cuh"

namespace dspark {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32, kHold = 8;

struct Fresh {
    int q0, n, ctx;
};

__device__ __forceinline__ Fresh request_of(const InsertScaledParams &p, int b, unsigned &flags)
{
    const int q0 = __ldg(p.query_start + b), q1 = __ldg(p.query_start + b + 1), ctx = __ldg(p.context_lens + b);
    Fresh r{q0, q1 - q0, ctx};
    if (q0 < 0 || q1 < q0 || q1 > p.num_rows || ctx < 0 ||
        (q1 > q0 && (int64_t)ctx + (q1 - q0) > p.table_blocks * p.block_size)) {
        flags |= kFlagLength;
        r.n = 0;
    }
    return r;
}

__device__ __forceinline__ int pages_of(const Fresh &r, int bs)
{
    return r.n ? (r.ctx + r.n - 1) / bs - r.ctx / bs + 1 : 0;
}

// max of |x| over the finite ones of a bf16 pair, by their bits
__device__ __forceinline__ uint32_t top2(uint32_t top, uint32_t w)
{
    w &= 0x7fff7fffu;
    return __vmaxu2(top, w & ~__vcmpgeu2(w, 0x7f807f80u));
}

__device__ __forceinline__ int exponent_of(uint32_t bits)  // of the largest |x|, as bf16 bits
{
    const int e = (int)(bits >> 7) - 127 - 8 + ((bits & 0x7fu) > 0x60u);
    return min(max(e, kScaleMin), kScaleMax);
}

// eight values times s as codes
__device__ __forceinline__ uint2 encode8(const uint4 &v, float s)
{
    const uint64_t s2 = pr(s, s);
    return make_uint2(e4m3x4(mul2(bf2_to_f2(v.x), s2), mul2(bf2_to_f2(v.y), s2)),
                      e4m3x4(mul2(bf2_to_f2(v.z), s2), mul2(bf2_to_f2(v.w), s2)));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 8) insert_scaled_kernel(const __grid_constant__ InsertScaledParams p)
{
    constexpr int kW = D / 4;  // 16-byte words of a token's K and V of a head: the same word for all of a thread's tokens
    static_assert(kThreads % kW == 0, "a thread keeps to K or to V");
    __shared__ int64_t scratch[kWarps + 4];
    __shared__ uint32_t tops[2][kWarps][2];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, H = p.num_kv_heads, bs = p.block_size;
    unsigned flags = 0;
    const attn::Find f = attn::find_request<kThreads>(
        p.num_requests, scratch, [&](int b) { return (int64_t)pages_of(request_of(p, b, flags), bs) * H; });
    const attn::Shares shares(f.total, gridDim.x);
    if (f.b >= 0) {
        int b = f.b;
        unsigned ignore = 0;
        Fresh r = request_of(p, b, ignore);
        const int64_t u0 = shares.start(blockIdx.x), u1 = shares.start(blockIdx.x + 1);
        int64_t of = u0 - f.before;  // the unit's number in its request
        int turn = 0;
        const int w = tid % kW, part = w >= kW / 2;
        for (int64_t u = u0; u < u1; u++, of++) {
            while (of >= (int64_t)pages_of(r, bs) * H) {
                of -= (int64_t)pages_of(r, bs) * H;
                r = request_of(p, ++b, ignore);
            }
            const int pi = (int)(of / H), h = (int)(of - (int64_t)pi * H), blk = r.ctx / bs + pi;
            const int64_t first = (int64_t)blk * bs;
            const int lo = pi ? (int)first : r.ctx, hi = (int)min((int64_t)r.ctx + r.n, first + bs);
            const int held = pi ? 0 : r.ctx - (int)first;  // the context's tokens in the page
            const int64_t page = __ldg(p.table + b * p.table_stride + blk);
            if (page < 0 || page >= p.num_blocks) {
                flags |= kFlagBlockRange;
                continue;
            }
            int8_t *scale = p.scales + (page * H + h) * 2;
            const int was0 = held ? page_exponent(p.scales, page, H, h, 0) : kScaleMin;
            const int was1 = held ? page_exponent(p.scales, page, H, h, 1) : kScaleMin;
            const uint16_t *src = (part ? p.v + h * p.v_hs : p.k + h * p.k_hs) + (w - part * (kW / 2)) * 8;
            const int64_t ts = part ? p.v_ts : p.k_ts;
            const int row0 = r.q0 + lo - r.ctx, rows = hi - lo, step = kThreads / kW;
            uint4 v[kHold];
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < kHold; k++) {
                const int x = tid / kW + k * step;
                v[k] = x < rows ? __ldg(reinterpret_cast<const uint4 *>(src + (row0 + x) * ts)) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < kHold; k++)
                top = top2(top2(top2(top2(top, v[k].x), v[k].y), v[k].z), v[k].w);
            for (int x = tid / kW + kHold * step; x < rows; x += step) {
                const uint4 y = __ldg(reinterpret_cast<const uint4 *>(src + (row0 + x) * ts));
                top = top2(top2(top2(top2(top, y.x), y.y), y.z), y.w);
            }
            top = max(top & 0xffffu, top >> 16);
            const uint32_t tk = __reduce_max_sync(0xffffffffu, part ? 0u : top), tv = __reduce_max_sync(0xffffffffu, part ? top : 0u);
            if (lane == 0)
                tops[turn][warp][0] = tk, tops[turn][warp][1] = tv;
            __syncthreads();  // everyone has read the old scale too
            uint32_t most[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < kWarps; i++)
                most[0] = max(most[0], tops[turn][i][0]), most[1] = max(most[1], tops[turn][i][1]);
            turn ^= 1;
            const int e0 = max(exponent_of(most[0]), was0), e1 = max(exponent_of(most[1]), was1);
            // the codes of the context's tokens in the page, where the scale grows: 16 bytes have one part
            unsigned char *cache = p.cache + ((page * H + h) * bs) * (int64_t)(2 * D);
            if (held && (e0 > was0 || e1 > was1))
                for (int x = tid; x < held * (D / 8); x += kThreads) {
                    const int d = x % (D / 8) >= D / 16 ? e1 - was1 : e0 - was0;
                    uint4 *at = reinterpret_cast<uint4 *>(cache + (int64_t)x * 16);
                    if (d)
                        *at = scale_codes(*at, half2_power(d));
                }
            if (tid == 0)
                scale[0] = (int8_t)e0, scale[1] = (int8_t)e1;
            const float s = __int_as_float((127 - (part ? e1 : e0)) << 23);
            unsigned char *dst = cache + (int64_t)(lo - first) * (2 * D) + w * 8;
#pragma unroll
            for (int k = 0; k < kHold; k++) {
                const int x = tid / kW + k * step;
                if (x < rows)
                    *reinterpret_cast<uint2 *>(dst + (int64_t)x * (2 * D)) = encode8(v[k], s);
            }
            for (int x = tid / kW + kHold * step; x < rows; x += step)
                *reinterpret_cast<uint2 *>(dst + (int64_t)x * (2 * D)) =
                    encode8(__ldg(reinterpret_cast<const uint4 *>(src + (row0 + x) * ts)), s);
        }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && lane == 0 && p.error_flags)
        atomicOr(p.error_flags, flags);
}

}  // namespace

cudaError_t launch_insert_scaled(const InsertScaledParams &p, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    const int64_t units = p.num_rows * p.num_kv_heads;  // at most: a page each
    const int ctas = (int)(units < 8 * (int64_t)sms ? units : 8 * (int64_t)sms);
    switch (p.head_dim) {
    case 64: return launch_pdl(insert_scaled_kernel<64>, ctas, kThreads, 0, stream, p);
    case 128: return launch_pdl(insert_scaled_kernel<128>, ctas, kThreads, 0, stream, p);
    default: return launch_pdl(insert_scaled_kernel<256>, ctas, kThreads, 0, stream, p);
    }
}

}  // namespace dspark
