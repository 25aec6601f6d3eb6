// kda_attn_prefill_e2m1.cu -- the prefill attention kernels over a 4-bit cache (a translation unit of their own, compiled
// beside the others').
#define KDA_PREFILL_E2M1
#include "kda_attn_prefill.cu"
