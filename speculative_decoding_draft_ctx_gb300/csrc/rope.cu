// sm_103a kernels of the cos|sin table and of rotary positions with the K/V
// insert.
//
// Defining passages: DSpark context-KV writer page, module docstring (partial
// NeoX RoPE from a cos|sin cache, the cache layout, fp8 of x / scale, slots
// < 0 not written); DSpark draft model page (the cos_sin_cache whose last dim
// is rotary_dim).  The interleaved pairing and the scaled frequencies are the
// usual forms those pages do not use.
//
// Table.  The angle p f of a far position in fp32 loses the turn it is in.
// Here the frequency is a 64-bit fixed-point fraction F = f / 2 pi * 2^64 of a
// turn, so p F mod 2^64 is the angle's fraction of a turn, exact but for F's
// own rounding (p 2^-65 turns): the wrap of the integer product is the range
// reduction.  The top bits give the nearest quarter turn, the signed rest (at
// most 1/8 turn) goes to fp32 with a relative rounding and through
// sincospif.  Bound: the store of 2 or 4 bytes per entry; a thread makes 4
// neighbouring angles, so it stores 8 or 16 bytes of cos and of sin.
//
// Rotation.  A head row of D dims is held by D / 8 lanes, 8 dims (16 bytes)
// each, so a warp takes 256 / D rows per step.  Half layout: the partner of
// dim i < r/2 is i + r/2, r/16 lanes away: one shuffle per word.
// Interleaved: both dims of a pair are in one lane.  Where a row is not
// 16-byte aligned, or r/2 is no whole number of lanes, the same code loads
// its elements and partners one by one (before any store of the warp, so in
// place is safe).  Per element the arithmetic is x1 c - x2 s in fp32 (the
// product of two bf16 values is exact there), rounded once to bf16.  Bound:
// the read and write of q and k.  A CTA walks (token, group of head rows)
// units; every lane issues kBatch rows' loads before it computes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ctx_kv_device.cuh"
#include "ctx_kv_internal.h"
#include "draft_attn_internal.h"

namespace dspark {
namespace {

// ------------------------------------------------------------------ the table

constexpr int kTableThreads = 256;

// cos and sin of 2 pi u 2^-64
__device__ __forceinline__ void turn_cos_sin(uint64_t u, float &c, float &s)
{
    const uint64_t quarter = (u + (1ull << 61)) >> 62;  // nearest quarter turn, 0..3 (4 wraps to 0)
    const int64_t rest = (int64_t)(u - (quarter << 62));  // in [-2^61, 2^61)
    // |rest| <= 1/8 turn; half turns = rest 2^-63
    float sn, cs;
    sincospif((float)rest * 0x1p-63f, &sn, &cs);
    const int n = (int)quarter & 3;
    const float a = (n & 1) ? sn : cs, b = (n & 1) ? cs : sn;
    c = (n == 1 || n == 2) ? -a : a;
    s = (n >= 2) ? -b : b;
}

// V entries per thread: 4 where r/2 is a multiple of 4 (whole 8- or 16-byte
// stores), else 1.
template <bool FP32, int V>
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ RopeTableParams p)
{
    pdl_enter();
    const int half = p.rotary_dim >> 1, per_row = half / V;
    const int64_t units = p.count * per_row;
    for (int64_t u = (int64_t)blockIdx.x * kTableThreads + threadIdx.x; u < units;
         u += (int64_t)gridDim.x * kTableThreads) {
        const int64_t row = u / per_row;
        const int i0 = (int)(u - row * per_row) * V;
        const uint64_t pos = (uint64_t)(p.first + row);
        float c[V], s[V];
#pragma unroll
        for (int j = 0; j < V; j++) {
            turn_cos_sin(pos * p.turns[i0 + j], c[j], s[j]);
            c[j] *= p.amplitude;
            s[j] *= p.amplitude;
        }
        const int64_t at = row * p.rotary_dim + i0;
        if constexpr (FP32) {
            float *o = static_cast<float *>(p.out) + at;
            if constexpr (V == 4) {
                *reinterpret_cast<float4 *>(o) = make_float4(c[0], c[1], c[2], c[3]);
                *reinterpret_cast<float4 *>(o + half) = make_float4(s[0], s[1], s[2], s[3]);
            } else {
                o[0] = c[0];
                o[half] = s[0];
            }
        } else {
            uint16_t *o = static_cast<uint16_t *>(p.out) + at;
            if constexpr (V == 4) {
                *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]));
                *reinterpret_cast<uint2 *>(o + half) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
            } else {
                o[0] = (uint16_t)pack_bf16x2(c[0], 0.0f);
                o[half] = (uint16_t)pack_bf16x2(s[0], 0.0f);
            }
        }
    }
}

// ------------------------------------------------------------------ the rotation

constexpr int kThreads = 256, kWarps = kThreads / 32, kBatch = 4;
constexpr unsigned kFlagSlot = 0x1u, kFlagPos = 0x2u;

__device__ __forceinline__ float bfl(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bfh(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// eight bf16 values from an address of any 2-byte alignment
__device__ __forceinline__ uint4 gather8(const uint16_t *p)
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
        w[j] = (uint32_t)p[2 * j] | ((uint32_t)p[2 * j + 1] << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// VEC: rows are 16-byte aligned and a lane's 8 dims rotate together (half
// layout: r % 16 == 0; interleaved: r % 8 == 0).
template <int D, bool VEC, bool TF32>
__global__ void __launch_bounds__(kThreads) rope_insert_kernel(const __grid_constant__ RopeInsertParams p)
{
    constexpr int L = D / 8, RPW = 32 / L;  // lanes per row, rows per warp step
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int q = lane % L, sub = lane / L;
    const int r = p.rotary_dim, half = r >> 1;
    const int Hq = p.num_heads, Hkv = p.num_kv_heads;
    const bool insert = p.slot_mapping != nullptr;
    const int rows = Hq + Hkv + (insert ? Hkv : 0);  // head rows of a token: q, k and (insert) v
    const int step = RPW * kWarps * gridDim.y;       // rows between two of a warp's row groups
    // the lane's first dim; the dims its rotation pairs with
    const int d0 = 8 * q;
    const int lanes_half = r >> 4;                   // VEC, half layout: lanes of one half
    Fp8Scale kq, vq;
    if (insert && p.fp8) {
        kq = fp8_scale(p.k_scale ? __ldg(p.k_scale) : 1.0f);
        vq = fp8_scale(p.v_scale ? __ldg(p.v_scale) : 1.0f);
    }
    const float sign = p.inverse ? -1.0f : 1.0f;
    unsigned flags = 0;

    for (int64_t t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
        int64_t pos = __ldg(p.positions + t);
        int64_t slot = insert ? __ldg(p.slot_mapping + t) : -1;
        const bool turn = pos >= 0 && pos < p.max_pos;
        if (!turn) {
            flags |= kFlagPos;
            slot = -1;
            pos = 0;
        }
        if (slot >= p.capacity) {
            flags |= kFlagSlot;
            slot = -1;
        }
        // cos and signed sin of the lane's dims: out = x c + partner s
        float c[8], s[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int d = d0 + e;
            c[e] = 1.0f, s[e] = 0.0f;
            if (turn && d < r) {
                const int i = p.interleaved ? d >> 1 : (d < half ? d : d - half);
                const bool upper = p.interleaved ? (d & 1) : d >= half;
                float sv;
                if constexpr (TF32) {
                    const float *cs = static_cast<const float *>(p.cos_sin) + pos * r;
                    c[e] = __ldg(cs + i), sv = __ldg(cs + half + i);
                } else {
                    const uint16_t *cs = static_cast<const uint16_t *>(p.cos_sin) + pos * r;
                    c[e] = __uint_as_float((uint32_t)__ldg(cs + i) << 16);
                    sv = __uint_as_float((uint32_t)__ldg(cs + half + i) << 16);
                }
                s[e] = (upper ? sv : -sv) * sign;
            }
        }
        const int64_t blk = slot >= 0 ? slot / p.block_size : 0;
        const int64_t row0 = slot >= 0 ? (blk * Hkv * p.block_size + (slot - blk * p.block_size)) * (2 * D) : 0;
        const int64_t hstride = (int64_t)p.block_size * (2 * D);

        for (int g = (blockIdx.y * kWarps + warp) * RPW; g < rows; g += step * kBatch) {
            uint4 x[kBatch];
            uint32_t partner[kBatch][VEC ? 1 : 4];
#pragma unroll
            for (int b = 0; b < kBatch; b++) {
                const int hh = g + b * step + sub;
                x[b] = make_uint4(0, 0, 0, 0);
                if (hh < rows) {
                    const uint16_t *src = hh < Hq         ? p.q + t * p.q_ts + hh * p.q_hs
                                          : hh < Hq + Hkv ? p.k + t * p.k_ts + (hh - Hq) * p.k_hs
                                                          : p.v + t * p.v_ts + (hh - Hq - Hkv) * p.v_hs;
                    if constexpr (VEC) {
                        x[b] = *reinterpret_cast<const uint4 *>(src + d0);
                    } else {
                        x[b] = gather8(src + d0);
                        if (hh < Hq + Hkv) {
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                uint32_t w = 0;
#pragma unroll
                                for (int e = 0; e < 2; e++) {
                                    const int d = d0 + 2 * j + e;
                                    int m = p.interleaved ? d ^ 1 : (d < half ? d + half : d - half);
                                    m = d < r ? m : d;
                                    w |= (uint32_t)src[m] << (16 * e);
                                }
                                partner[b][j] = w;
                            }
                        }
                    }
                }
            }
            if constexpr (!VEC)
                __syncwarp();  // in place: every partner is read before any row of the batch is written
#pragma unroll
            for (int b = 0; b < kBatch; b++) {
                const int hh = g + b * step + sub;
                if (g + b * step >= rows)
                    break;  // uniform over the warp
                uint32_t w[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
                uint32_t y[4];
                if (hh < Hq + Hkv || VEC) {  // VEC: every lane takes part in the shuffles
                    uint32_t pw[4];
                    if constexpr (VEC) {
                        if (p.interleaved) {
#pragma unroll
                            for (int j = 0; j < 4; j++)
                                pw[j] = (w[j] >> 16) | (w[j] << 16);
                        } else {
                            const int pl = q < lanes_half ? lane + lanes_half : q < 2 * lanes_half ? lane - lanes_half : lane;
#pragma unroll
                            for (int j = 0; j < 4; j++)
                                pw[j] = __shfl_sync(0xffffffffu, w[j], pl);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            pw[j] = partner[b][j];
                    }
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        float lo = bfl(w[j]), hi = bfh(w[j]);
                        if (d0 + 2 * j < r) {
                            lo = fmaf(lo, c[2 * j], bfl(pw[j]) * s[2 * j]);
                            hi = fmaf(hi, c[2 * j + 1], bfh(pw[j]) * s[2 * j + 1]);
                        }
                        y[j] = d0 + 2 * j < r && turn ? pack_bf16x2(lo, hi) : w[j];
                    }
                }
                if (hh >= rows)
                    continue;
                if (hh < Hq + Hkv) {
                    uint16_t *dst = hh < Hq ? p.q_out + t * p.qo_ts + hh * p.qo_hs
                                            : p.k_out + t * p.ko_ts + (hh - Hq) * p.ko_hs;
                    if constexpr (VEC) {
                        *reinterpret_cast<uint4 *>(dst + d0) = make_uint4(y[0], y[1], y[2], y[3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            dst[d0 + 2 * j] = (uint16_t)y[j];
                            dst[d0 + 2 * j + 1] = (uint16_t)(y[j] >> 16);
                        }
                    }
                }
                if (slot >= 0 && hh >= Hq) {
                    const bool is_k = hh < Hq + Hkv;
                    const uint4 o = is_k ? make_uint4(y[0], y[1], y[2], y[3]) : x[b];
                    const int64_t at = row0 + (is_k ? hh - Hq : hh - Hq - Hkv) * hstride + (is_k ? 0 : D) + d0;
                    if (p.fp8)
                        *reinterpret_cast<uint2 *>(p.cache + at) = quantise8(o, is_k ? kq : vq);
                    else
                        *reinterpret_cast<uint4 *>(p.cache + 2 * at) = o;
                }
            }
        }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && lane == 0 && p.error_flags)
        atomicOr(p.error_flags, flags);
}

int sm_count(cudaError_t &e)
{
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

cudaError_t launch_grid(void (*kernel)(RopeInsertParams), const RopeInsertParams &p, int blocks, int splits,
                        cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)splits);
    cfg.blockDim = dim3((unsigned)kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D>
cudaError_t launch_rope_d(const RopeInsertParams &p, cudaStream_t stream)
{
    cudaError_t e;
    const int sms = sm_count(e);
    if (e != cudaSuccess)
        return e;
    // One CTA per token while tokens last for four CTAs per SM; fewer tokens
    // split their head rows over blockIdx.y so that the small calls of a draft
    // step have one batch of loads per warp.
    const int rows = p.num_heads + p.num_kv_heads * (p.slot_mapping ? 2 : 1);
    const int groups = (rows + 256 / D * kWarps - 1) / (256 / D * kWarps);
    const int most = 4 * sms;
    const int blocks = (int)(p.num_tokens < most ? p.num_tokens : most);
    int splits = most / (blocks > 0 ? blocks : 1);
    splits = splits < 1 ? 1 : splits > groups ? groups : splits;
    if (splits > 64)
        splits = 64;
    if (p.vec)
        return launch_grid(p.table_fp32 ? rope_insert_kernel<D, true, true> : rope_insert_kernel<D, true, false>, p,
                           blocks, splits, stream);
    return launch_grid(p.table_fp32 ? rope_insert_kernel<D, false, true> : rope_insert_kernel<D, false, false>, p,
                       blocks, splits, stream);
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableParams &p, bool fp32, cudaStream_t stream)
{
    cudaError_t e;
    const int sms = sm_count(e);
    if (e != cudaSuccess)
        return e;
    const int v = (p.rotary_dim >> 1) % 4 == 0 ? 4 : 1;
    const int64_t units = p.count * ((p.rotary_dim >> 1) / v);
    const int64_t want = (units + kTableThreads - 1) / kTableThreads;
    const int blocks = (int)(want < 8 * sms ? want : 8 * sms);
    if (v == 4)
        return launch_pdl(fp32 ? rope_table_kernel<true, 4> : rope_table_kernel<false, 4>, blocks, kTableThreads, 0,
                          stream, p);
    return launch_pdl(fp32 ? rope_table_kernel<true, 1> : rope_table_kernel<false, 1>, blocks, kTableThreads, 0,
                      stream, p);
}

cudaError_t launch_rope_insert(const RopeInsertParams &p, int head_dim, cudaStream_t stream)
{
    switch (head_dim) {
    case 64: return launch_rope_d<64>(p, stream);
    case 128: return launch_rope_d<128>(p, stream);
    case 256: return launch_rope_d<256>(p, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dspark
