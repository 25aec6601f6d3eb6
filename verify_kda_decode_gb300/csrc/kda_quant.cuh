// kda_quant.cuh -- rounding to the codes that a key-value cache holds: E4M3, and E2M1 with an E4M3 scale for each 16
// elements (kda_kv.cu, kda_rope.cu).
#pragma once

#include "kda_internal.cuh"
#include "kda_tc.cuh"

namespace kda {

// A scale and its correctly rounded reciprocal, NaN where quotients cannot be had from it.
__device__ __forceinline__ float2 with_reciprocal(float scale)
{
    const float a = fabsf(scale);
    return make_float2(scale, a > 1e-18f && a < 1e18f ? __frcp_rn(scale) : NAN);
}

// (rarely called: kept out of the callers' code)
static __device__ __noinline__ float quotient(float a, float b) { return __fdiv_rn(a, b); }

// q = -g / scale.x, the IEEE quotients, of eight elements' negatives; `scale` from with_reciprocal.
// Markstein's theorem gives that quotient from the correctly rounded reciprocal: q = f r, then q + (f - q scale) r, three
// packed operations for two elements (a division each took 57 us for 33000 tokens to E4M3, bound by its instructions);
// with f = -g as q - (q scale + g) r, whose inner sum is +0 where q is exact, so that a zero keeps its sign.  Infinities,
// and scales whose reciprocal or products could leave the normal range (their reciprocal is given as NaN), take the
// division.
__device__ __forceinline__ void neg_quotients8(const float *g, float2 scale, float *q)
{
    float t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float e0, e1;
        tc::mul2(q[i], q[i + 1], g[i], g[i + 1], -scale.y, -scale.y);
        tc::fma2(e0, e1, q[i], q[i + 1], scale.x, scale.x, g[i], g[i + 1]);
        tc::fma2(q[i], q[i + 1], e0, e1, -scale.y, -scale.y, q[i], q[i + 1]);
        tc::add2(t0, t1, t0, t1, q[i], q[i + 1]);
    }
    if (!(fabsf(t0 + t1) < 1e30f)) {
#pragma unroll
        for (int i = 0; i < 8; i++) q[i] = quotient(-g[i], scale.x);
    }
}

// Eight E4M3 codes, to the nearest, clamped to +-448; NaN stays NaN.
__device__ __forceinline__ uint2 e4m3x8(const float *q)
{
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
        o[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]), __NV_SATFINITE, __NV_E4M3) |
               (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
    return make_uint2(o[0], o[1]);
}

// Eight E2M1 codes, the first in the lowest bits, to the nearest (ties to the even code), clamped to +-6.
__device__ __forceinline__ uint32_t e2m1x8(const float *q)
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}

// Largest magnitude of eight elements, as bits (which order magnitudes, with infinity above them and NaN above that).
__device__ __forceinline__ uint32_t magnitude8(const float *y)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) m = max(m, __float_as_uint(y[i]) & 0x7fffffffu);
    return m;
}

// The E4M3 scale of a block whose largest magnitude has these bits: a sixth of it (6 is the largest code), to the nearest,
// from the least code 2^-9 (so that small blocks keep what 4 bits can) to 448; NaN for a block with a NaN.
__device__ __forceinline__ uint32_t block_scale(uint32_t magnitude)
{
    return max(1u, (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(magnitude), 6.f), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ float2 block_scale_value(uint32_t code)
{
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
    return make_float2(s, __frcp_rn(s));
}

}  // namespace kda
