// kda_attn_common.cuh -- what the decode and prefill attention kernels share: which keys the new
// tokens of a sequence see, and the order of the tiles that cover them.
#pragma once

#include "kda_paged.cuh"

namespace kda {

constexpr float kLn2 = 0.693147180559945309f;

// Keys that tokens at positions [p0, p1] (p1 >= p0) of a row of `len` tokens see, as tiles of kTile
// keys: tiles [0, st) hold the sinks, then tiles from `first` to the last one needed.  A token at p
// sees j <= p with p - j < W or j < S (W = INT_MAX without a window, S then 0).
template <int kTile>
struct KeyRange {
    int end;     // keys below `end` only
    int lo;      // ... and from `lo` on, or below S
    int st, first, count;
    __device__ __forceinline__ KeyRange(int p0, int p1, int len, int W, int S)
    {
        end = max(0, min(len, p1 + 1));
        const long long l = (long long)p0 - W + 1;
        lo = (int)max(0ll, min((long long)end, l));
        first = lo / kTile;
        st = min((min(S, end) + kTile - 1) / kTile, first);
        count = st + (end + kTile - 1) / kTile - first;
    }
    __device__ __forceinline__ int tile(int i) const { return i < st ? i : i - st + first; }
};

__device__ __forceinline__ bool key_visible(int j, int p, int W, int S) { return j <= p && (p - j < W || j < S); }

// The two 16-bit types of queries and outputs, and of the weights P that multiply the values.  The running maximum's
// key has the weight 2^kShift, and the maximum is moved when a score passes it by more than kGrow (powers of two).
// bfloat16 has FP32's range.  Halves are normal from 2^-14 to below 2^16: with the maximum at 2^11 .. 2^15 a weight keeps
// its relative precision of 2^-11 down to 2^-25 of the largest one, and below that is off by at most 2^-36 of it.  (With the
// maximum at 1 .. 2^8, 32768 keys 2^-25 under a sink were off by 5 to 30 times the output's rounding.)
struct Half {
    static constexpr bool is_half = true;
    static constexpr float kShift = 11.f, kGrow = 4.f;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
struct Bf16 {
    static constexpr bool is_half = false;
    static constexpr float kShift = 0.f, kGrow = 8.f;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// Four E4M3 codes -> four halves in order; exact.
__device__ __forceinline__ void e4m3x4_half4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

// What scores are multiplied with: 0 as the least that keeps hidden scores at -inf.  A NaN (of a scale in the cache) stays one.
__device__ __forceinline__ float score_scale(float x) { return x < 1e-37f ? 1e-37f : x; }

// With an E4M3 cache the products are taken in halves.  A bfloat16 row of queries is brought to a maximum in
// [1, 2) by a power of two first (exact but for elements under 2^-14 of it, whose error stays under 2^-25 of
// it): `mag` is the row's largest magnitude's bits; returns the factor `down` for the elements and `up` for
// the scores.  Rows with infinities or NaN stay as they are.
__device__ __forceinline__ void query_scale(uint32_t mag, float &down, float &up)
{
    const int ex = (int)(mag >> 7);                              // biased exponent
    const int e = ex == 255 ? 0 : min(max(ex, 1) - 127, 126);
    down = __uint_as_float((uint32_t)(127 - e) << 23);
    up = __uint_as_float((uint32_t)max(127 + e, 1) << 23);
}
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, const uint4 &x)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t y = (&x.x)[i];
        m = max(m, max(y & 0x7fffu, (y >> 16) & 0x7fffu));
    }
    return m;
}
// Eight bfloat16 -> eight halves, times `down`.
__device__ __forceinline__ uint4 scaled_halves(const uint4 &x, float down)
{
    uint4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t y = (&x.x)[i];
        (&r.x)[i] = Half::pack(__uint_as_float(y << 16) * down, __uint_as_float(y & 0xffff0000u) * down);
    }
    return r;
}

template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

}  // namespace kda
