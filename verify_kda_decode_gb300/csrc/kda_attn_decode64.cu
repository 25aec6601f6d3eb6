// kda_attn_decode64.cu -- the decode attention kernels for head_dim 64 (a translation unit of their own, compiled beside
// the other's).
#include "kda_attn_decode.cuh"

namespace kda {

size_t attn_decode_workspace(int D) { return Partials::kCounters * sizeof(int) + 2 * kMaxCtas * Partials::slot_floats(D) * sizeof(float); }

cudaError_t launch_attn_decode64(const AttnParams &p, cudaStream_t stream) { return launch_types<64>(p, stream); }

}  // namespace kda
