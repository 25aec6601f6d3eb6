// kda_paged_api.cu -- the extern "C" entry points of the paged key-value cache and its attention:
// argument checks, then kernel launches.  As in kda_api.cu nothing is allocated, synchronised
// (except kda_kv_get_error) or read from device memory on the host.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "kda_paged.cuh"

void kda_set_last_error(const char *msg);

namespace {

kda_status fail(kda_status s, const char *fmt, ...)
{
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    kda_set_last_error(msg);
    return s;
}

kda_status launched(cudaError_t e)
{
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "CUDA: %s", cudaGetErrorString(e));
    kda_set_last_error("");
    return KDA_OK;
}

bool aligned(const void *p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

#define NEED(p, n)                                                                                                  \
    do {                                                                                                            \
        if (!aligned(p, n)) return fail(KDA_ERR_INVALID_ARG, "%s is null or not %d-byte aligned", #p, (int)(n)); \
    } while (0)
#define CHECK(expr)                          \
    do {                                     \
        kda_status s_ = (expr);              \
        if (s_ != KDA_OK) return s_;         \
    } while (0)

kda_status check_cache(const kda_kv_cache *cache)
{
    if (!cache) return fail(KDA_ERR_INVALID_ARG, "cache is null");
    if (cache->kv_dtype != KDA_T_BF16 && cache->kv_dtype != KDA_T_F16 && cache->kv_dtype != KDA_T_E4M3)
        return fail(KDA_ERR_INVALID_ARG, "kv_dtype=%d is none of KDA_T_BF16, KDA_T_F16, KDA_T_E4M3", cache->kv_dtype);
    if (cache->num_layers < 1 || cache->num_pages < 1 || cache->num_kv_heads < 1 || cache->rows < 1 || cache->max_pages < 1)
        return fail(KDA_ERR_INVALID_ARG, "num_layers=%d, num_pages=%d, num_kv_heads=%d, rows=%d, max_pages=%d: each must be >= 1",
                    cache->num_layers, cache->num_pages, cache->num_kv_heads, cache->rows, cache->max_pages);
    if (cache->num_kv_heads > 4096) return fail(KDA_ERR_INVALID_ARG, "num_kv_heads=%d > 4096", cache->num_kv_heads);
    if (cache->page_size != 16 && cache->page_size != 32 && cache->page_size != 64 && cache->page_size != 128)
        return fail(KDA_ERR_UNSUPPORTED, "page_size=%d: only 16, 32, 64 and 128 are built", cache->page_size);
    if (cache->head_dim != 64 && cache->head_dim != 128)
        return fail(KDA_ERR_UNSUPPORTED, "head_dim=%d: only 64 and 128 are built", cache->head_dim);
    if (cache->rows > kda::kMaxRows) return fail(KDA_ERR_UNSUPPORTED, "rows=%d: at most %d", cache->rows, kda::kMaxRows);
    if ((long long)cache->rows * cache->max_pages > 0x7fffffffll)
        return fail(KDA_ERR_UNSUPPORTED, "rows * max_pages = %lld does not fit 31 bits", (long long)cache->rows * cache->max_pages);
    if ((long long)cache->max_pages * cache->page_size > 0x3fffffffll)
        return fail(KDA_ERR_UNSUPPORTED, "max_pages * page_size = %lld tokens: at most 2^30 - 1", (long long)cache->max_pages * cache->page_size);
    if (cache->num_pages > 0x3fffffff) return fail(KDA_ERR_UNSUPPORTED, "num_pages=%d: at most 2^30 - 1", cache->num_pages);
    NEED(cache->k, 16);
    NEED(cache->v, 16);
    NEED(cache->page_table, 4);
    NEED(cache->seq_lens, 4);
    NEED(cache->page_refs, 4);
    NEED(cache->err_word, 4);
    if (cache->kv_dtype == KDA_T_E4M3) {
        NEED(cache->k_scale, 4);
        NEED(cache->v_scale, 4);
    }
    return KDA_OK;
}

kda::PagedCache paged(const kda_kv_cache *cache)
{
    kda::PagedCache c;
    c.k = static_cast<uint8_t *>(cache->k);
    c.v = static_cast<uint8_t *>(cache->v);
    c.dtype = cache->kv_dtype;
    c.layers = cache->num_layers;
    c.pages = cache->num_pages;
    c.Hkv = cache->num_kv_heads;
    c.ps = cache->page_size;
    c.ps_log2 = 0;
    while (1 << c.ps_log2 < c.ps) c.ps_log2++;
    c.D = cache->head_dim;
    c.rows = cache->rows;
    c.width = cache->max_pages;
    c.table = cache->page_table;
    c.lens = cache->seq_lens;
    c.refs = cache->page_refs;
    c.k_scale = cache->k_scale;
    c.v_scale = cache->v_scale;
    c.err = cache->err_word;
    return c;
}

kda_status check_distinct_rows(const kda_kv_cache *cache, int32_t B)
{
    if (B < 0) return fail(KDA_ERR_INVALID_ARG, "B=%d < 0", B);
    if (B > cache->rows) return fail(KDA_ERR_INVALID_ARG, "B=%d exceeds rows=%d (rows must be distinct)", B, cache->rows);
    return KDA_OK;
}

kda_status check_kv_workspace(const kda_kv_cache *cache, const void *workspace, size_t bytes)
{
    NEED(workspace, 256);
    const size_t need = kda_kv_workspace_size(cache);
    if (bytes < need) return fail(KDA_ERR_INVALID_ARG, "workspace_bytes=%zu < %zu", bytes, need);
    return KDA_OK;
}

kda_status check_layer_index(const kda_kv_cache *cache, int32_t layer)
{
    if (layer < 0 || layer >= cache->num_layers)
        return fail(KDA_ERR_INVALID_ARG, "layer=%d outside [0, %d)", layer, cache->num_layers);
    return KDA_OK;
}

// Layout of [seq, token, head, D] elements, D contiguous, read 16 bytes at a time.
kda_status check_layout(const kda_kv_cache *cache, const kda_tokens_layout *l, const char *name)
{
    if (!l) return fail(KDA_ERR_INVALID_ARG, "layout of %s is null", name);
    if (l->dtype != KDA_T_BF16 && l->dtype != KDA_T_F16)
        return fail(KDA_ERR_INVALID_ARG, "%s: dtype=%d is neither KDA_T_BF16 nor KDA_T_F16", name, l->dtype);
    if (cache->kv_dtype != KDA_T_E4M3 && l->dtype != cache->kv_dtype)
        return fail(KDA_ERR_INVALID_ARG, "%s: dtype=%d, the cache holds %d", name, l->dtype, cache->kv_dtype);
    if (l->seq_stride < 0 || l->token_stride < 0 || l->head_stride < 0) return fail(KDA_ERR_INVALID_ARG, "%s: negative stride", name);
    if ((l->seq_stride | l->token_stride | l->head_stride) & 7)
        return fail(KDA_ERR_INVALID_ARG, "%s: strides %lld, %lld, %lld are not all multiples of 8 elements", name,
                    (long long)l->seq_stride, (long long)l->token_stride, (long long)l->head_stride);
    return KDA_OK;
}

kda::TokensLayout layout(const kda_tokens_layout *l) { return {l->seq_stride, l->token_stride, l->head_stride}; }

kda_status check_attn(const kda_kv_cache *cache, int32_t layer, const kda_attn_desc *desc)
{
    CHECK(check_cache(cache));
    CHECK(check_layer_index(cache, layer));
    if (!desc) return fail(KDA_ERR_INVALID_ARG, "desc is null");
    if (desc->num_q_heads < 1 || desc->num_q_heads % cache->num_kv_heads)
        return fail(KDA_ERR_INVALID_ARG, "num_q_heads=%d is no multiple of num_kv_heads=%d", desc->num_q_heads, cache->num_kv_heads);
    if (desc->num_q_heads / cache->num_kv_heads > kda::kMaxGroup)
        return fail(KDA_ERR_UNSUPPORTED, "num_q_heads=%d: more than %d per kv head", desc->num_q_heads, kda::kMaxGroup);
    if (!isfinite(desc->scale) || desc->scale < 0.f) return fail(KDA_ERR_INVALID_ARG, "scale must be finite and >= 0");
    if (desc->window < 0 || desc->sinks < 0) return fail(KDA_ERR_INVALID_ARG, "window=%d, sinks=%d: each must be >= 0", desc->window, desc->sinks);
    return check_layout(cache, &desc->q, "q");
}

kda_status check_attn_workspace(const kda_kv_cache *cache, const void *workspace, size_t bytes)
{
    NEED(workspace, 256);
    const size_t need = kda_attn_workspace_size(cache);
    if (bytes < need) return fail(KDA_ERR_INVALID_ARG, "workspace_bytes=%zu < %zu", bytes, need);
    return KDA_OK;
}

kda::AttnParams attn_params(const kda_kv_cache *cache, int32_t layer, const kda_attn_desc *desc, const int32_t *rows,
                            int32_t B, int32_t T, const void *q, void *out, float *lse, void *workspace)
{
    kda::AttnParams p;
    memset(&p, 0, sizeof p);
    p.c = paged(cache);
    p.layer = layer;
    p.Hq = desc->num_q_heads;
    p.G = desc->num_q_heads / cache->num_kv_heads;
    p.scale_log2 = desc->scale * 1.44269504088896341f;
    p.window = desc->window;
    p.sinks = desc->sinks;
    p.rows = rows;
    p.B = B;
    p.T = T;
    p.q = static_cast<const uint16_t *>(q);
    p.ql = layout(&desc->q);
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.f16 = desc->q.dtype == KDA_T_F16;
    p.ws = static_cast<uint8_t *>(workspace);
    return p;
}

kda::KvCall kv_call(const kda_kv_cache *cache, const int32_t *rows, const int32_t *arg, int32_t B, void *workspace)
{
    kda::KvCall p;
    memset(&p, 0, sizeof p);
    p.c = paged(cache);
    p.rows = rows;
    p.arg = arg;
    p.B = B;
    p.ws = static_cast<int *>(workspace);
    return p;
}

}  // namespace

extern "C" {

size_t kda_kv_workspace_size(const kda_kv_cache *cache)
{
    if (!cache || cache->rows < 1 || cache->num_pages < 1) return 0;
    return kda::kv_workspace_ints(cache->rows, cache->num_pages) * sizeof(int);
}

kda_status kda_kv_extend(const kda_kv_cache *cache, const int32_t *rows, const int32_t *n_tokens, int32_t n_all,
                         int32_t B, void *workspace, size_t workspace_bytes, void *stream)
{
    CHECK(check_cache(cache));
    CHECK(check_distinct_rows(cache, B));
    if (!n_tokens && n_all < 0) return fail(KDA_ERR_INVALID_ARG, "n_all=%d < 0", n_all);
    if (B == 0) return launched(cudaSuccess);
    NEED(rows, 4);
    if (n_tokens) NEED(n_tokens, 4);
    CHECK(check_kv_workspace(cache, workspace, workspace_bytes));
    kda::KvCall p = kv_call(cache, rows, n_tokens, B, workspace);
    p.uniform = n_all;
    return launched(kda::launch_kv_extend(p, static_cast<cudaStream_t>(stream)));
}

kda_status kda_kv_truncate(const kda_kv_cache *cache, const int32_t *rows, const int32_t *new_lens, int32_t B,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    CHECK(check_cache(cache));
    CHECK(check_distinct_rows(cache, B));
    if (B == 0) return launched(cudaSuccess);
    NEED(rows, 4);
    NEED(new_lens, 4);
    CHECK(check_kv_workspace(cache, workspace, workspace_bytes));
    return launched(kda::launch_kv_truncate(kv_call(cache, rows, new_lens, B, workspace), static_cast<cudaStream_t>(stream)));
}

kda_status kda_kv_fork(const kda_kv_cache *cache, const int32_t *src_rows, const int32_t *dst_rows, int32_t n,
                       void *workspace, size_t workspace_bytes, void *stream)
{
    CHECK(check_cache(cache));
    CHECK(check_distinct_rows(cache, n));
    if (n == 0) return launched(cudaSuccess);
    NEED(src_rows, 4);
    NEED(dst_rows, 4);
    CHECK(check_kv_workspace(cache, workspace, workspace_bytes));
    return launched(kda::launch_kv_fork(kv_call(cache, dst_rows, src_rows, n, workspace), static_cast<cudaStream_t>(stream)));
}

kda_status kda_kv_compact(const kda_kv_cache *cache, int32_t *remap, void *workspace, size_t workspace_bytes, void *stream)
{
    CHECK(check_cache(cache));
    NEED(remap, 4);
    CHECK(check_kv_workspace(cache, workspace, workspace_bytes));
    kda::KvCall p = kv_call(cache, nullptr, nullptr, 0, workspace);
    p.remap = remap;
    return launched(kda::launch_kv_compact(p, static_cast<cudaStream_t>(stream)));
}

kda_status kda_kv_append(const kda_kv_cache *cache, int32_t layer, const int32_t *rows, int32_t B, int32_t T,
                         const int32_t *n_tokens, const int32_t *cu_seqlens, const void *k,
                         const kda_tokens_layout *k_layout, const void *v, const kda_tokens_layout *v_layout, void *stream)
{
    CHECK(check_cache(cache));
    CHECK(check_layer_index(cache, layer));
    if (B < 0 || T < 0) return fail(KDA_ERR_INVALID_ARG, "B=%d, T=%d: each must be >= 0", B, T);
    CHECK(check_layout(cache, k_layout, "k"));
    CHECK(check_layout(cache, v_layout, "v"));
    if (k_layout->dtype != v_layout->dtype) return fail(KDA_ERR_INVALID_ARG, "k and v have different types");
    if (n_tokens && cu_seqlens) return fail(KDA_ERR_INVALID_ARG, "n_tokens and cu_seqlens exclude each other");
    if (!cu_seqlens && (long long)B * T > 0x7fffffffll) return fail(KDA_ERR_UNSUPPORTED, "B * T = %lld does not fit 31 bits", (long long)B * T);
    if (B == 0 || T == 0) return launched(cudaSuccess);
    NEED(rows, 4);
    if (n_tokens) NEED(n_tokens, 4);
    if (cu_seqlens) NEED(cu_seqlens, 4);
    NEED(k, 16);
    NEED(v, 16);
    kda::AppendParams p;
    memset(&p, 0, sizeof p);
    p.c = paged(cache);
    p.layer = layer;
    p.rows = rows;
    p.n_tokens = n_tokens;
    p.cu = cu_seqlens;
    p.B = B;
    p.T = T;
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.kl = layout(k_layout);
    p.vl = layout(v_layout);
    p.f16 = k_layout->dtype == KDA_T_F16;
    return launched(kda::launch_kv_append(p, static_cast<cudaStream_t>(stream)));
}

size_t kda_attn_workspace_size(const kda_kv_cache *cache)
{
    if (!cache || (cache->head_dim != 64 && cache->head_dim != 128)) return 0;
    const size_t a = kda::attn_decode_workspace(cache->head_dim), b = kda::attn_prefill_workspace(cache->head_dim);
    return a > b ? a : b;
}

kda_status kda_attn_decode(const kda_kv_cache *cache, int32_t layer, const kda_attn_desc *desc, const int32_t *rows,
                           int32_t B, int32_t T, const int32_t *n_tokens, const void *q, void *out, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    CHECK(check_attn(cache, layer, desc));
    if (B < 0) return fail(KDA_ERR_INVALID_ARG, "B=%d < 0", B);
    if (B > 65535) return fail(KDA_ERR_UNSUPPORTED, "B=%d > 65535", B);
    if (T < 1 || T > kda::kMaxAttnT) return fail(KDA_ERR_INVALID_ARG, "T=%d outside [1, %d]", T, kda::kMaxAttnT);
    if (B == 0) return launched(cudaSuccess);
    NEED(rows, 4);
    if (n_tokens) NEED(n_tokens, 4);
    NEED(q, 16);
    NEED(out, 16);
    if (lse) NEED(lse, 4);
    CHECK(check_attn_workspace(cache, workspace, workspace_bytes));
    kda::AttnParams p = attn_params(cache, layer, desc, rows, B, T, q, out, lse, workspace);
    p.n_tokens = n_tokens;
    return launched(p.c.D == 64 ? kda::launch_attn_decode64(p, static_cast<cudaStream_t>(stream))
                               : kda::launch_attn_decode128(p, static_cast<cudaStream_t>(stream)));
}

kda_status kda_attn_prefill(const kda_kv_cache *cache, int32_t layer, const kda_attn_desc *desc, const int32_t *rows,
                            int32_t B, const int32_t *cu_seqlens, int32_t total_tokens, int32_t max_len, const void *q,
                            void *out, float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    CHECK(check_attn(cache, layer, desc));
    if (B < 0) return fail(KDA_ERR_INVALID_ARG, "B=%d < 0", B);
    if (B > 65535) return fail(KDA_ERR_UNSUPPORTED, "B=%d > 65535", B);
    if (total_tokens < 0) return fail(KDA_ERR_INVALID_ARG, "total_tokens=%d < 0", total_tokens);
    if (max_len < 0) return fail(KDA_ERR_INVALID_ARG, "max_len=%d < 0", max_len);
    if (B == 0 || total_tokens == 0) return launched(cudaSuccess);
    if (max_len == 0) return fail(KDA_ERR_INVALID_ARG, "max_len=0 with total_tokens=%d > 0", total_tokens);
    if ((long long)total_tokens * (desc->num_q_heads / cache->num_kv_heads) > 0x3fffffffll)
        return fail(KDA_ERR_UNSUPPORTED, "total_tokens=%d with %d query heads per kv head: at most 2^30 - 1 rows", total_tokens,
                    desc->num_q_heads / cache->num_kv_heads);
    NEED(rows, 4);
    NEED(cu_seqlens, 4);
    NEED(q, 16);
    NEED(out, 16);
    if (lse) NEED(lse, 4);
    CHECK(check_attn_workspace(cache, workspace, workspace_bytes));
    kda::AttnParams p = attn_params(cache, layer, desc, rows, B, max_len, q, out, lse, workspace);
    p.cu = cu_seqlens;
    p.total = total_tokens;
    return launched(kda::launch_attn_prefill(p, static_cast<cudaStream_t>(stream)));
}

kda_status kda_kv_get_error(const kda_kv_cache *cache, int32_t *host_err, void *stream)
{
    if (!cache || !cache->err_word || !host_err) return fail(KDA_ERR_INVALID_ARG, "null argument");
    kda_pool pool;
    memset(&pool, 0, sizeof pool);
    pool.err_word = cache->err_word;
    return kda_get_error(&pool, host_err, stream);
}

}  // extern "C"
