// The weight accumulation by head dim and cache type.
#include "attn_weight.cuh"

namespace dspark {

cudaError_t launch_attention_weight(const AttnParams &p, int head_dim, bool fp8, cudaStream_t stream)
{
    switch (head_dim) {
    case 64: return fp8 ? attn::weight<64, true>(p, stream) : attn::weight<64, false>(p, stream);
    case 128: return fp8 ? attn::weight<128, true>(p, stream) : attn::weight<128, false>(p, stream);
    default: return fp8 ? attn::weight<256, true>(p, stream) : attn::weight<256, false>(p, stream);
    }
}

}  // namespace dspark
