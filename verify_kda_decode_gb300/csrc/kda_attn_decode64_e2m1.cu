// kda_attn_decode64_e2m1.cu -- the decode attention kernels for head_dim 64 over a 4-bit cache (a translation unit of their own,
// compiled beside the others').
#include "kda_attn_decode.cuh"

namespace kda {

cudaError_t launch_attn_decode64_e2m1(const AttnParams &p, cudaStream_t stream) { return launch_types<64, kKvE2M1>(p, stream); }

}  // namespace kda
