// kda_attn_decode64.cu -- the decode attention kernels for head_dim 64 (a translation unit of their own, compiled beside
// the other's).
#include "kda_attn_decode.cuh"

namespace kda {

size_t attn_decode_workspace(int D) { return Partials::kCounters * sizeof(int) + 2 * kMaxCtas * Partials::slot_floats(D) * sizeof(float); }

cudaError_t launch_attn_decode64(const AttnParams &p, cudaStream_t stream) 
{
    return p.c.dtype == KDA_T_E2M1   ? launch_attn_decode64_e2m1(p, stream)
           : p.c.dtype == KDA_T_E4M3 ? launch_types<64, kKvE4M3>(p, stream)
                                     : launch_types<64, kKv16>(p, stream);
}

}  // namespace kda
