// kda_attn_decode128.cu -- the decode attention kernels for head_dim 128 (a translation unit of their own, compiled beside
// the other's).
#include "kda_attn_decode.cuh"

namespace kda {

cudaError_t launch_attn_decode128(const AttnParams &p, cudaStream_t stream) 
{
    return p.c.dtype == KDA_T_E2M1   ? launch_attn_decode128_e2m1(p, stream)
           : p.c.dtype == KDA_T_E4M3 ? launch_types<128, kKvE4M3>(p, stream)
                                     : launch_types<128, kKv16>(p, stream);
}

}  // namespace kda
