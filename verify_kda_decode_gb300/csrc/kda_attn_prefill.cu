#include "kda_paged.cuh"
namespace kda {
size_t attn_prefill_workspace(int) { return 0; }
cudaError_t launch_attn_prefill(const AttnParams &, cudaStream_t) { return cudaErrorNotSupported; }
}
