// kda_attn_decode128.cu -- the decode attention kernels for head_dim 128 (a translation unit of their own, compiled beside
// the other's).
#include "kda_attn_decode.cuh"

namespace kda {

cudaError_t launch_attn_decode128(const AttnParams &p, cudaStream_t stream) { return launch_types<128>(p, stream); }

}  // namespace kda
