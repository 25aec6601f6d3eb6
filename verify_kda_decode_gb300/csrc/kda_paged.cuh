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
    // bytes of one token of one head (E2M1: its codes and block scales, which stand apart, see kda_kv_cache)
    __host__ __device__ int token_bytes() const { return dtype == KDA_T_E2M1 ? D / 2 + D / 16 : dtype == KDA_T_E4M3 ? D : 2 * D; }
    // bytes of one page of one layer, all heads
    __host__ __device__ size_t page_bytes() const { return (size_t)Hkv * ps * token_bytes(); }
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

// How positions turn the pairs of a head (kda_rope_desc).
struct Turns {
    const unsigned long long *freq;   // [rot / 2] turns per position, in units of 2^-64
    int rot, adjacent;
    float scale;
};
// A tensor whose heads are turned on their way from src to dst.
struct TurnedTensor {
    const uint16_t *src;
    uint16_t *dst;
    int heads;
    TokensLayout sl, dl;
};
struct RopeParams {
    Turns r;
    const int *pos;                // [tokens]
    int tokens, T, D;              // T: tokens per sequence
    int lanes_log2;                // lanes of a head, parts: warps of a token (set by the launcher)
    int parts;
    TurnedTensor x[2];
    bool f16;
};
cudaError_t launch_rope(RopeParams p, cudaStream_t stream);

// An append whose keys (and the queries `q`, where it has heads) are turned, or one to a 4-bit cache.
struct AppendTurnParams {
    AppendParams a;
    Turns r;                       // freq null: nothing is turned
    TurnedTensor q;
    int parts;
};
cudaError_t launch_kv_append_turn(AppendTurnParams p, cudaStream_t stream);

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
cudaError_t launch_attn_decode64_e2m1(const AttnParams &p, cudaStream_t stream);
cudaError_t launch_attn_decode128_e2m1(const AttnParams &p, cudaStream_t stream);
cudaError_t launch_attn_prefill(const AttnParams &p, cudaStream_t stream);
cudaError_t launch_attn_prefill_e2m1(const AttnParams &p, cudaStream_t stream);
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

// Position, and page, of token `tok` of an append (token in_seq of sequence seq without offsets), looked up by a whole warp;
// false where it has none (`say` is the thread that sets the error word then).
__device__ __forceinline__ bool append_place(const AppendParams &p, long long tok, long long seq, long long in_seq, int lane, bool say,
                                             int &pos, int &page)
{
    const PagedCache &c = p.c;
    int b, t, n;
    if (p.cu) {
        // the sequence whose offsets hold this row: the last b with cu[b] <= tok, 32 at a time
        int a = 0, e = p.B;   // in [a, e)
        while (e - a > 1) {
            const int step = (e - a + 31) / 32;
            const int at = a + lane * step;
            const bool le = at < e && p.cu[at] <= tok;
            const unsigned m = __ballot_sync(~0u, le);
            const int k = m ? 31 - __clz(m) : 0;
            a += k * step;
            e = min(e, a + step);
        }
        b = a;
        const int c0 = p.cu[b], c1 = p.cu[b + 1];
        if (c0 < 0 || c1 < c0 || c1 > p.T) {
            if (say) atomicOr(c.err, KDA_DEVERR_SEQLEN);
            return false;
        }
        if (tok < c0 || tok >= c1) return false;   // rows outside every sequence
        t = (int)(tok - c0);
        n = c1 - c0;
    } else {
        b = (int)seq;
        t = (int)in_seq;
        n = p.n_tokens ? p.n_tokens[b] : p.T;
    }
    const SeqInfo s = seq_info(c, p.rows[b], n, p.cu ? 0x7fffffff : p.T, t == 0 && say);
    if (!s.ok || t >= n) return false;
    if (n > s.len) {   // fewer tokens in the row than the call brings
        if (say) atomicOr(c.err, KDA_DEVERR_SEQLEN);
        return false;
    }
    pos = s.len - n + t;
    page = c.table[(size_t)s.row * c.width + (pos >> c.ps_log2)];
    if ((unsigned)page >= (unsigned)c.pages) {
        if (say) atomicOr(c.err, KDA_DEVERR_PAGE);
        return false;
    }
    return true;
}

}  // namespace kda
