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

// The two 16-bit types of queries and outputs.
struct Half {
    static constexpr bool is_half = true;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
struct Bf16 {
    static constexpr bool is_half = false;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// Two E4M3 codes (low half first) -> two halves; exact.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t w, int hi)
{
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(hi ? w >> 16 : w & 0xffffu), __NV_E4M3);
    return (uint32_t)r.x | ((uint32_t)r.y << 16);
}
// ... -> two values of the query's type; exact in both.
template <typename Q>
__device__ __forceinline__ uint32_t e4m3x2_as(uint32_t w, int hi)
{
    const uint32_t h = e4m3x2_half2(w, hi);
    if constexpr (Q::is_half) return h;
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return Bf16::pack(f.x, f.y);
}

template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

}  // namespace kda
