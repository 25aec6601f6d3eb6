// kda_paged.cuh -- the paged key-value cache as the kernels see it, and the launchers of the
// kernels that work on it (kda_kv.cu, kda_attn_decode.cuh, kda_attn_prefill.cu).
#pragma once

#include "kda_internal.cuh"
#include "kda_ptx.cuh"

namespace kda {

constexpr int kMaxAttnT = 16;      // new tokens per sequence of a decode / verify call
constexpr int kMaxGroup = 64;      // query heads per key head
constexpr int kMaxRows = 1 << 18;  // rows of a page table

struct PagedCache {
    uint8_t *k, *v;                // [layers, pages, Hkv, ps, D]
    int dtype;                     // kda_elem_type
    int layers, pages, Hkv, ps, ps_log2, D;
    int rows, width;               // page table
    int *table, *lens, *refs;
    const float *k_scale, *v_scale;
    int *err;
    __host__ __device__ int elem() const { return dtype == KDA_T_E4M3 ? 1 : 2; }
    // bytes of one page of one layer, all heads
    __host__ __device__ size_t page_bytes() const { return (size_t)Hkv * ps * D * elem(); }
};

struct KvCall {
    PagedCache c;
    const int *rows, *arg;         // arg: n_tokens / new_lens / src_rows
    int uniform, B;
    int lanes;                     // threads of an entry (set by the launcher)
    int *ws;                       // see kv_workspace_ints
    int *remap;
};

// Scratch of the page calls, in ints: counters, seven arrays of `rows`, two lists of page ids.
constexpr int kKvMeta = 16, kKvRowArrays = 7;
inline size_t kv_workspace_ints(int rows, int pages) { return kKvMeta + (size_t)kKvRowArrays * rows + 2 * (size_t)pages; }

cudaError_t launch_kv_extend(const KvCall &p, cudaStream_t stream);
cudaError_t launch_kv_truncate(KvCall p, cudaStream_t stream);
cudaError_t launch_kv_fork(KvCall p, cudaStream_t stream);
cudaError_t launch_kv_compact(const KvCall &p, cudaStream_t stream);

struct TokensLayout { long long seq, token, head; };   // strides in elements

struct AppendParams {
    PagedCache c;
    int layer;
    const int *rows, *n_tokens, *cu;
    int B, T;                      // T: tokens per sequence, or all packed tokens with cu
    const uint16_t *k, *v;
    TokensLayout kl, vl;
    bool f16;                      // 16-bit inputs are half, not bfloat16
};
cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream);

struct AttnParams {
    PagedCache c;
    int layer, Hq, G;
    float scale_log2;              // scale * log2(e)
    int window, sinks;
    const int *rows, *n_tokens, *cu;
    int B, T;                      // decode: tokens per sequence; prefill: bound on a sequence's tokens
    int total;                     // prefill: packed tokens
    float inv_g;                   // prefill: 1 / G (set by the launcher)
    const uint16_t *q;
    TokensLayout ql;
    uint16_t *out;
    float *lse;
    bool f16;
    uint8_t *ws;
};
// The attention workspace begins with counters (int, all 0 between calls), which both kernels use, then
// holds partial results.
constexpr size_t kAttnCounters = 4096;
cudaError_t launch_attn_decode64(const AttnParams &p, cudaStream_t stream);
cudaError_t launch_attn_decode128(const AttnParams &p, cudaStream_t stream);
cudaError_t launch_attn_prefill(const AttnParams &p, cudaStream_t stream);
size_t attn_decode_workspace(int D);
size_t attn_prefill_workspace(int D);

// SMs of the current device, kept per device ordinal.
inline cudaError_t paged_sm_count(int *sms)
{
    static std::atomic<int> cache[KernelSetup::kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= KernelSetup::kMaxDevices) return cudaErrorInvalidDevice;
    int n = cache[dev].load(std::memory_order_acquire);
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        cache[dev].store(n, std::memory_order_release);
    }
    *sms = n;
    return cudaSuccess;
}

// launch_pdl with clusters of `cluster` CTAs.
template <typename Kern, typename Arg>
cudaError_t launch_pdl_cluster(Kern kern, dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t stream, const Arg &arg)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, arg);
}

// What a sequence of a call asks for: its row, length and new tokens; `ok` is false (and the
// error word is set by the thread with `report`) where they do not fit the cache.
struct SeqInfo {
    int row, len, n;
    bool ok;
};
__device__ __forceinline__ SeqInfo seq_info(const PagedCache &c, int row, int n, int n_max, bool report)
{
    SeqInfo s;
    s.row = row;
    s.n = n;
    s.len = 0;
    int err = 0;
    if ((unsigned)row >= (unsigned)c.rows) err = KDA_DEVERR_SLOT;
    else if (n < 0 || n > n_max) err = KDA_DEVERR_TOKENS;
    else {
        s.len = c.lens[row];
        if (s.len < 0 || (long long)s.len > (long long)c.width << c.ps_log2) err = KDA_DEVERR_SEQLEN;
    }
    s.ok = err == 0;
    if (err && report) atomicOr(c.err, err);
    return s;
}

}  // namespace kda
