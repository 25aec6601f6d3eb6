// kda_kv.cu -- pages of the key-value cache: extend, truncate, fork, compact, append.
//
// The page calls work on small integer arrays (a table row per sequence, a count per page) and
// have to give the same ids whatever order their threads run in.  Ids come from ranks: the r-th
// page asked for gets the r-th free id, both ranks exclusive prefix sums over fixed orders, so no
// result depends on an atomic's order (the atomics add to counts or set flags).
#include <cooperative_groups.h>

#include "kda_paged.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

// Where new ids are given out (extend, compact) one cluster of eight CTAs does the bookkeeping: 8192 threads that can meet at a cluster
// barrier, against one CTA's 1024 (a scan of 64 Ki counts reads 8 per thread instead of 64) and
// against a grid that would need a launch for each phase.
constexpr int kCl = 8, kNt = 1024, kAll = kCl * kNt;
constexpr size_t kMaxMaps = 3 * (kMaxRows / 32) * 4;   // bytes of the row maps of the largest table

struct ScanMem {
    int2 warp[32];
    int2 total;    // this CTA's sums, read by the others through distributed shared memory
};

// Exclusive prefix sums of two numbers over all threads of the cluster in order (CTA rank, thread);
// every thread gets its prefixes and the totals.  Ends with a barrier, so `sm` can be used again.
__device__ int2 cluster_scan(cg::cluster_group &cl, ScanMem &sm, int2 v, int2 &total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int2 x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(~0u, x.x, o), b = __shfl_up_sync(~0u, x.y, o);
        if (lane >= o) x.x += a, x.y += b;
    }
    if (lane == 31) sm.warp[w] = x;
    __syncthreads();
    if (w == 0) {
        int2 y = sm.warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(~0u, y.x, o), b = __shfl_up_sync(~0u, y.y, o);
            if (lane >= o) y.x += a, y.y += b;
        }
        sm.warp[lane] = y;
        if (lane == 31) sm.total = y;
    }
    __syncthreads();
    int2 before = make_int2(x.x - v.x, x.y - v.y);
    if (w) before.x += sm.warp[w - 1].x, before.y += sm.warp[w - 1].y;
    cl.sync();
    int2 all = make_int2(0, 0);
    const int me = (int)cl.block_rank();
#pragma unroll
    for (int r = 0; r < kCl; r++) {
        const int2 t = *cl.map_shared_rank(&sm.total, r);
        if (r < me) before.x += t.x, before.y += t.y;
        all.x += t.x, all.y += t.y;
    }
    total = all;
    cl.sync();   // every CTA has read the totals
    return before;
}

struct Scratch {
    int *meta, *off, *want, *have, *flag, *cow_src, *cow_dst, *cow_n, *list, *list2;
    __device__ explicit Scratch(const KvCall &p)
    {
        const int R = p.c.rows;
        meta = p.ws;
        off = p.ws + kKvMeta;
        want = off + R;
        have = want + R;
        flag = have + R;
        cow_src = flag + R;
        cow_dst = cow_src + R;
        cow_n = cow_dst + R;
        list = cow_n + R;
        list2 = list + p.c.pages;
    }
};

__device__ __forceinline__ int ceil_pages(const PagedCache &c, int len) { return (int)(((long long)len + c.ps - 1) >> c.ps_log2); }

// Which rows a call names, and which it names more than once, as bit maps in shared memory that every
// CTA makes for itself (no exchange between CTAs).  With `sources`, also which rows p.arg names.
struct RowMaps {
    uint32_t *once, *twice, *source;
    __device__ RowMaps(const KvCall &p, uint32_t *smem, bool sources)
    {
        const int words = (p.c.rows + 31) / 32;
        once = smem;
        twice = once + words;
        source = twice + words;
        for (int i = threadIdx.x; i < words * (sources ? 3 : 2); i += kNt) smem[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < p.B; i += kNt) {
            const int r = p.rows[i];
            if ((unsigned)r < (unsigned)p.c.rows) {
                const uint32_t bit = 1u << (r & 31);
                if (atomicOr(&once[r >> 5], bit) & bit) atomicOr(&twice[r >> 5], bit);
            }
            if (sources) {
                const int q = p.arg[i];
                if ((unsigned)q < (unsigned)p.c.rows) atomicOr(&source[q >> 5], 1u << (q & 31));
            }
        }
        __syncthreads();
    }
    // in range and named once
    __device__ bool good(const PagedCache &c, int r) const { return (unsigned)r < (unsigned)c.rows && !(twice[r >> 5] >> (r & 31) & 1); }
    __device__ bool is_source(int r) const { return source[r >> 5] >> (r & 31) & 1; }
};
inline size_t row_maps_bytes(const KvCall &p, bool sources) { return (size_t)((p.c.rows + 31) / 32) * 4 * (sources ? 3 : 2); }

__global__ void __launch_bounds__(kNt, 1) kda_kv_extend_kernel(const KvCall p)
{
    extern __shared__ uint32_t maps[];
    __shared__ ScanMem sm;
    cg::cluster_group cl = cg::this_cluster();
    const PagedCache &c = p.c;
    const Scratch s(p);
    const int g = (int)cl.block_rank() * kNt + threadIdx.x;
    grid_dependency_wait();
    if (g == 0) s.meta[0] = 0;   // pages to copy, for the kernel that follows
    const RowMaps rows(p, maps, false);
    // what each entry asks for, and how many pages are free: their places in the order of the call and of the ids
    const int per = (p.B + kAll - 1) / kAll;
    int mine = 0;
    for (int i = g * per; i < min(p.B, (g + 1) * per); i++) {
        const int r = p.rows[i], n = p.arg ? p.arg[i] : p.uniform;
        int err = 0, want = 0, copy = 0, have = 0;
        if (!rows.good(c, r)) err = KDA_DEVERR_SLOT;
        else if (n < 0) err = KDA_DEVERR_TOKENS;
        else {
            const int len = c.lens[r];
            if (len < 0 || (long long)len > (long long)c.width << c.ps_log2) err = KDA_DEVERR_SEQLEN;
            else if ((long long)len + n > (long long)c.width << c.ps_log2) err = KDA_DEVERR_NOPAGES;
            else {
                have = ceil_pages(c, len);
                if (n > 0 && (len & (c.ps - 1))) {
                    const int tail = c.table[(size_t)r * c.width + have - 1];
                    if ((unsigned)tail >= (unsigned)c.pages) err = KDA_DEVERR_PAGE;
                    else copy = c.refs[tail] > 1;
                }
                if (!err) want = ceil_pages(c, len + n) - have + copy;
            }
        }
        if (err) atomicOr(c.err, err);
        s.want[i] = want;
        s.have[i] = have;
        s.flag[i] = err ? 4 : copy;
        mine += want;
    }
    const int cp = (c.pages + kAll - 1) / kAll, lo = min(c.pages, g * cp), hi = min(c.pages, lo + cp);
    int free_here = 0;
    for (int q = lo; q < hi; q++) free_here += c.refs[q] == 0;
    int2 sums;
    const int2 before = cluster_scan(cl, sm, make_int2(mine, free_here), sums);
    const int total = sums.x, n_free = sums.y;
    int at = before.x, rank = before.y;
    for (int i = g * per; i < min(p.B, (g + 1) * per); i++) {
        s.off[i] = at;
        at += s.want[i];
    }
    // the lowest free ids, as many as are asked for
    if (free_here && rank < total)
        for (int q = lo; q < hi; q++)
            if (c.refs[q] == 0) {
                if (rank < total) s.list[rank] = q;
                rank++;
            }
    cl.sync();
    // lengths and copied pages of the entries that fit
    for (int i = g; i < p.B; i += kAll) {
        const int f = __ldcg(&s.flag[i]), w = __ldcg(&s.want[i]);
        if (f & 4) continue;
        if (w > 0 && __ldcg(&s.off[i]) + (long long)w > n_free) {
            atomicOr(c.err, KDA_DEVERR_NOPAGES);
            continue;
        }
        const int r = p.rows[i], n = p.arg ? p.arg[i] : p.uniform;
        if (f & 1) {   // the copy of the shared last page comes first
            int *e = &c.table[(size_t)r * c.width + __ldcg(&s.have[i]) - 1];
            const int from = *e, to = __ldcg(&s.list[__ldcg(&s.off[i])]);
            const int slot = atomicAdd(&s.meta[0], 1);   // any order: the copies are independent
            s.cow_src[slot] = from;
            s.cow_dst[slot] = to;
            s.cow_n[slot] = c.lens[r] & (c.ps - 1);
            atomicSub(&c.refs[from], 1);
            c.refs[to] = 1;
            *e = to;
        }
        c.lens[r] += n;
    }
    // the added pages, one thread each: the entry by bisection over the offsets
    for (int t = g; t < min(total, n_free); t += kAll) {
        int a = 0, b = p.B - 1;   // the last entry whose offset is <= t
        while (a < b) {
            const int m = (a + b + 1) >> 1;
            if (__ldcg(&s.off[m]) <= t) a = m;
            else b = m - 1;
        }
        const int f = __ldcg(&s.flag[a]), o = __ldcg(&s.off[a]), j = t - o - (f & 1);
        if ((f & 4) || j < 0 || o + (long long)__ldcg(&s.want[a]) > n_free) continue;
        const int page = __ldcg(&s.list[t]);
        c.table[(size_t)p.rows[a] * c.width + __ldcg(&s.have[a]) + j] = page;
        c.refs[page] = 1;
    }
}

// Copies the filled tokens of the shared pages that extend replaced, in every layer: 2 KiB pieces of a
// head's tokens, a warp each with four 16-byte loads a lane in flight (a warp for a head's whole run of
// tokens took 20 us for 64 copies of up to 64 tokens, 4 heads, 4 layers; its loads waited for one another).
// Most calls have none, and the count is read first.
constexpr int kTail = 2048;
__global__ void __launch_bounds__(256) kda_kv_copy_tails_kernel(const KvCall p)
{
    const PagedCache &c = p.c;
    const Scratch s(p);
    grid_dependency_wait();
    const int n = s.meta[0], lane = threadIdx.x & 31;
    const size_t row = (size_t)c.D * c.elem(), head = row * c.ps;
    const int pieces = (int)((head + kTail - 1) / kTail);
    const long long items = (long long)n * c.layers * 2 * c.Hkv * pieces;
    for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (long long)gridDim.x * 8) {
        long long x = it;
        const int piece = (int)(x % pieces);
        x /= pieces;
        const int h = (int)(x % c.Hkv);
        x /= c.Hkv;
        const int kv = (int)(x & 1);
        x >>= 1;
        const int layer = (int)(x % c.layers), i = (int)(x / c.layers);
        const int chunks = (int)(s.cow_n[i] * row) / 16 - piece * (kTail / 16);   // left from this piece on
        uint8_t *base = (kv ? c.v : c.k) + (size_t)layer * c.pages * c.page_bytes() + h * head + (size_t)piece * kTail;
        const uint4 *src = reinterpret_cast<const uint4 *>(base + (size_t)s.cow_src[i] * c.page_bytes());
        uint4 *dst = reinterpret_cast<uint4 *>(base + (size_t)s.cow_dst[i] * c.page_bytes());
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; u++)
            if (lane + 32 * u < chunks) v[u] = __ldcs(src + lane + 32 * u);
#pragma unroll
        for (int u = 0; u < 4; u++)
            if (lane + 32 * u < chunks) __stcs(dst + lane + 32 * u, v[u]);
    }
}

// Threads of an entry of a call over n rows, in powers of two: a CTA's at most (so that a CTA barrier
// separates the reads of a row's length from its write), a warp at least.
inline int lanes_per_entry(int n)
{
    int l = kNt;
    while (l > 32 && (long long)l * n > 16 * kNt) l >>= 1;
    return l;
}
inline unsigned entry_ctas(int n) { return (unsigned)(((long long)n * lanes_per_entry(n) + kNt - 1) / kNt); }

__global__ void __launch_bounds__(kNt, 1) kda_kv_truncate_kernel(const KvCall p)
{
    extern __shared__ uint32_t maps[];
    const PagedCache &c = p.c;
    grid_dependency_wait();
    const RowMaps rows(p, maps, false);
    const int L = p.lanes, i = (int)(((long long)blockIdx.x * kNt + threadIdx.x) / L), lane = threadIdx.x & (L - 1);
    bool ok = false;
    int r = 0, keep = 0, have = 0, nl = 0;
    if (i < p.B) {
        int err = 0;
        r = p.rows[i];
        if (!rows.good(c, r)) err = KDA_DEVERR_SLOT;
        else {
            nl = p.arg[i];
            const int len = c.lens[r];
            if (nl < 0 || nl > len || (long long)len > (long long)c.width << c.ps_log2) err = KDA_DEVERR_SEQLEN;
            else {
                keep = ceil_pages(c, nl);
                have = ceil_pages(c, len);
                ok = true;
            }
        }
        if (err && lane == 0) atomicOr(c.err, err);
    }
    __syncthreads();   // every lane has read its row's length
    if (!ok) return;
    int *t = c.table + (size_t)r * c.width;
    for (int j = keep + lane; j < have; j += L) {
        const int page = t[j];
        if ((unsigned)page < (unsigned)c.pages) atomicSub(&c.refs[page], 1);
        else atomicOr(c.err, KDA_DEVERR_PAGE);
        t[j] = -1;
    }
    if (lane == 0) c.lens[r] = nl;
}

__global__ void __launch_bounds__(kNt, 1) kda_kv_fork_kernel(const KvCall p)
{
    extern __shared__ uint32_t maps[];
    const PagedCache &c = p.c;
    grid_dependency_wait();
    const RowMaps rows(p, maps, true);
    const int L = p.lanes, i = (int)(((long long)blockIdx.x * kNt + threadIdx.x) / L), lane = threadIdx.x & (L - 1);
    bool ok = false;
    int dst = 0, src = 0, old_pages = 0, new_pages = 0, len = 0;
    if (i < p.B) {
        int err = 0;
        src = p.arg[i];
        dst = p.rows[i];
        if (!rows.good(c, dst) || (unsigned)src >= (unsigned)c.rows || rows.is_source(dst)) err = KDA_DEVERR_SLOT;
        else {
            len = c.lens[src];
            const int old = c.lens[dst];
            const long long most = (long long)c.width << c.ps_log2;
            if (len < 0 || len > most || old < 0 || old > most) err = KDA_DEVERR_SEQLEN;
            else {
                old_pages = ceil_pages(c, old);
                new_pages = ceil_pages(c, len);
                ok = true;
            }
        }
        if (err && lane == 0) atomicOr(c.err, err);
    }
    __syncthreads();   // every lane has read the lengths (a source is never a destination)
    if (!ok) return;
    int *td = c.table + (size_t)dst * c.width;
    const int *ts = c.table + (size_t)src * c.width;
    for (int j = lane; j < max(old_pages, new_pages); j += L) {
        int page = -1;
        if (j < old_pages) {
            const int q = td[j];
            if ((unsigned)q < (unsigned)c.pages) atomicSub(&c.refs[q], 1);
            else atomicOr(c.err, KDA_DEVERR_PAGE);
        }
        if (j < new_pages) {
            page = ts[j];
            if ((unsigned)page < (unsigned)c.pages) atomicAdd(&c.refs[page], 1);
            else atomicOr(c.err, KDA_DEVERR_PAGE);
        }
        td[j] = page;
    }
    if (lane == 0) c.lens[dst] = len;
}

// Which pages move where: the r-th page in use with an id >= n goes to the r-th free id < n
// (n = pages in use; there are as many of the one as of the other).
__global__ void __launch_bounds__(kNt, 1) kda_kv_compact_kernel(const KvCall p)
{
    __shared__ ScanMem sm;
    cg::cluster_group cl = cg::this_cluster();
    const PagedCache &c = p.c;
    const Scratch s(p);
    const int g = (int)cl.block_rank() * kNt + threadIdx.x;
    grid_dependency_wait();
    const int cp = (c.pages + kAll - 1) / kAll, lo = min(c.pages, g * cp), hi = min(c.pages, lo + cp);
    int live = 0;
    for (int q = lo; q < hi; q++) live += c.refs[q] != 0;
    int2 sums;
    cluster_scan(cl, sm, make_int2(live, 0), sums);
    const int n = sums.x;
    int high = 0, low = 0;
    for (int q = lo; q < hi; q++) {
        const bool used = c.refs[q] != 0;
        high += used && q >= n;
        low += !used && q < n;
    }
    const int2 before = cluster_scan(cl, sm, make_int2(high, low), sums);
    const int moves = sums.x;
    int rh = before.x, rl = before.y;
    for (int q = lo; q < hi; q++) {
        const bool used = c.refs[q] != 0;
        if (used && q >= n) s.list2[rh++] = q;
        else {
            if (!used && q < n) s.list[rl++] = q;
            p.remap[q] = used ? q : -1;
        }
    }
    if (g == 0) s.meta[0] = moves;
    cl.sync();
    for (int t = g; t < moves; t += kAll) {
        const int from = __ldcg(&s.list2[t]), to = __ldcg(&s.list[t]);
        p.remap[from] = to;
        c.refs[to] = c.refs[from];
        c.refs[from] = 0;
    }
}

// Moves the pages' data (whole pages of one layer are contiguous: 16 KiB pieces, 256 threads with
// four 16-byte loads each in flight) and renames the table's entries.
constexpr int kPiece = 256 * 16 * 4;
__global__ void __launch_bounds__(256) kda_kv_move_kernel(const KvCall p)
{
    const PagedCache &c = p.c;
    const Scratch s(p);
    grid_dependency_wait();
    const int n = s.meta[0], tid = threadIdx.x;
    const size_t bytes = c.page_bytes();
    const int pieces = (int)((bytes + kPiece - 1) / kPiece);
    const long long items = (long long)n * c.layers * 2 * pieces;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        long long x = it;
        const int piece = (int)(x % pieces);
        x /= pieces;
        const int kv = (int)(x & 1);
        x >>= 1;
        const int layer = (int)(x % c.layers), i = (int)(x / c.layers);
        uint8_t *base = (kv ? c.v : c.k) + (size_t)layer * c.pages * bytes + (size_t)piece * kPiece;
        const uint4 *src = reinterpret_cast<const uint4 *>(base + (size_t)s.list2[i] * bytes);
        uint4 *dst = reinterpret_cast<uint4 *>(base + (size_t)s.list[i] * bytes);
        const int chunks = (int)(min(bytes - (size_t)piece * kPiece, (size_t)kPiece) / 16);
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; u++)
            if (tid + u * 256 < chunks) v[u] = __ldcs(src + tid + u * 256);
#pragma unroll
        for (int u = 0; u < 4; u++)
            if (tid + u * 256 < chunks) __stcs(dst + tid + u * 256, v[u]);
    }
    if (n == 0) return;
    const long long entries = (long long)c.rows * c.width;
    for (long long e = (long long)blockIdx.x * 256 + tid; e < entries; e += (long long)gridDim.x * 256) {
        const int page = c.table[e];
        if ((unsigned)page < (unsigned)c.pages) {
            const int to = p.remap[page];
            if (to != page) c.table[e] = to;
        }
    }
}

// ---------------------------------------------------------------------------------- append

// One warp per new token: lanes over the token's 16-byte source pieces (8 elements), keys then
// values.  Pure data movement, bound by HBM for prompts and by the launch for a decode step.
template <bool E4M3, bool F16>
__device__ __forceinline__ void append_piece(const uint4 w, uint8_t *dst, float2 scale)   // scale and its reciprocal
{
    if constexpr (!E4M3) {
        *reinterpret_cast<uint4 *>(dst) = w;
    } else {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
        float g[8], q[8];   // g: the elements' negatives, for zeros' signs (below)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float2 v;
            if constexpr (F16) {
                const uint32_t y = x[i] ^ 0x80008000u;
                v = __half22float2(*reinterpret_cast<const __half2 *>(&y));
            } else {
                v = make_float2(__uint_as_float(x[i] << 16 ^ 0x80000000u), __uint_as_float((x[i] & 0xffff0000u) ^ 0x80000000u));
            }
            g[2 * i] = v.x;
            g[2 * i + 1] = v.y;
        }
        // The code is the rounding of the IEEE quotient.  Markstein's theorem gives that quotient from the correctly
        // rounded reciprocal: q = f r, then q + (f - q scale) r, three packed operations for two elements
        // (a division each took 57 us for 33000 tokens, bound by its instructions); with f = -g as q - (q scale + g) r,
        // whose inner sum is +0 where q is exact, so that a zero keeps its sign.  Infinities, and scales whose
        // reciprocal or products could leave the normal range (their reciprocal is given as NaN), take the
        // division.
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
            for (int i = 0; i < 8; i++) q[i] = __fdiv_rn(-g[i], scale.x);
        }
        uint32_t o[2];
#pragma unroll
        for (int i = 0; i < 2; i++)
            o[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]), __NV_SATFINITE, __NV_E4M3) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(o[0], o[1]);
    }
}

// A scale and its correctly rounded reciprocal, NaN where quotients cannot be had from it.
__device__ __forceinline__ float2 with_reciprocal(float scale)
{
    const float a = fabsf(scale);
    return make_float2(scale, a > 1e-18f && a < 1e18f ? __frcp_rn(scale) : NAN);
}

template <bool E4M3, bool F16>
__global__ void __launch_bounds__(256) kda_kv_append_kernel(const AppendParams p)
{
    constexpr int kScales = 64;   // key heads whose scales are kept on chip
    __shared__ float2 scales[2][E4M3 ? kScales : 1];
    const PagedCache &c = p.c;
    const int lane = threadIdx.x & 31;
    const long long tok = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long tokens = p.cu ? p.T : (long long)p.B * p.T;
    grid_dependency_wait();
    auto scale = [&](int kv, int h) {
        if constexpr (!E4M3) return make_float2(1.f, 1.f);
        else return h < kScales ? scales[kv][h] : with_reciprocal((kv ? c.v_scale : c.k_scale)[p.layer * c.Hkv + h]);
    };
    // The token's first pieces are on their way while its place is found, a chain of five loads (offsets, row,
    // length, page) that took longer than moving the data.
    const int per_log2 = c.D == 128 ? 4 : 3, pieces = c.Hkv << per_log2;   // 8 elements each
    const long long seq = p.cu ? 0 : tok / p.T, in_seq = tok - seq * p.T;
    const uint16_t *ks = p.k + (p.cu ? 0 : seq * p.kl.seq) + in_seq * p.kl.token, *vs = p.v + (p.cu ? 0 : seq * p.vl.seq) + in_seq * p.vl.token;
    constexpr int kAhead = 4;
    uint4 kw[kAhead], vw[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; a++) {
        const int q = lane + 32 * a, h = q >> per_log2, i = q & ((1 << per_log2) - 1);
        if (tok < tokens && q < pieces) {
            kw[a] = __ldcs(reinterpret_cast<const uint4 *>(ks + h * p.kl.head + i * 8));
            vw[a] = __ldcs(reinterpret_cast<const uint4 *>(vs + h * p.vl.head + i * 8));
        }
    }
    if constexpr (E4M3) {
        for (int i = threadIdx.x; i < 2 * min(c.Hkv, kScales); i += 256)
            scales[i & 1][i >> 1] = with_reciprocal(((i & 1) ? c.v_scale : c.k_scale)[p.layer * c.Hkv + (i >> 1)]);
        __syncthreads();
    }
    if (tok >= tokens) return;
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
            if (lane == 0) atomicOr(c.err, KDA_DEVERR_SEQLEN);
            return;
        }
        if (tok < c0 || tok >= c1) return;   // rows outside every sequence
        t = (int)(tok - c0);
        n = c1 - c0;
    } else {
        b = (int)seq;
        t = (int)in_seq;
        n = p.n_tokens ? p.n_tokens[b] : p.T;
    }
    const SeqInfo s = seq_info(c, p.rows[b], n, p.cu ? 0x7fffffff : p.T, t == 0 && lane == 0);
    if (!s.ok || t >= n) return;
    if (n > s.len) {   // fewer tokens in the row than the call brings
        if (lane == 0) atomicOr(c.err, KDA_DEVERR_SEQLEN);
        return;
    }
    const int pos = s.len - n + t;
    const int page = c.table[(size_t)s.row * c.width + (pos >> c.ps_log2)];
    if ((unsigned)page >= (unsigned)c.pages) {
        if (lane == 0) atomicOr(c.err, KDA_DEVERR_PAGE);
        return;
    }
    constexpr int ES = E4M3 ? 1 : 2;
    const size_t row = (size_t)c.D * ES, head = row * c.ps;
    const size_t at = ((size_t)p.layer * c.pages + page) * c.page_bytes() + (pos & (c.ps - 1)) * row;
    auto put = [&](int q, const uint4 &kx, const uint4 &vx) {
        const int h = q >> per_log2, i = q & ((1 << per_log2) - 1);
        const size_t to = at + h * head + (size_t)i * 8 * ES;
        append_piece<E4M3, F16>(kx, c.k + to, scale(0, h));
        append_piece<E4M3, F16>(vx, c.v + to, scale(1, h));
    };
#pragma unroll
    for (int a = 0; a < kAhead; a++)
        if (lane + 32 * a < pieces) put(lane + 32 * a, kw[a], vw[a]);
    for (int q = lane + 32 * kAhead; q < pieces; q += 32) {
        const int h = q >> per_log2, i = q & ((1 << per_log2) - 1);
        put(q, __ldcs(reinterpret_cast<const uint4 *>(ks + h * p.kl.head + i * 8)), __ldcs(reinterpret_cast<const uint4 *>(vs + h * p.vl.head + i * 8)));
    }
}

template <bool E4M3, bool F16>
cudaError_t append_as(const AppendParams &p, cudaStream_t stream)
{
    const long long tokens = p.cu ? p.T : (long long)p.B * p.T;
    return launch_pdl(kda_kv_append_kernel<E4M3, F16>, dim3((unsigned)((tokens + 7) / 8)), dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t launch_kv_extend(const KvCall &p, cudaStream_t stream)
{
    static KernelSetup setup;
    int sms = 0;
    const size_t smem = row_maps_bytes(p, false);
    cudaError_t e = paged_sm_count(&sms);
    if (e == cudaSuccess) e = setup.get(kda_kv_extend_kernel, kNt, kMaxMaps, 0, nullptr);
    if (e == cudaSuccess) e = launch_pdl_cluster(kda_kv_extend_kernel, dim3(kCl), dim3(kNt), smem, kCl, stream, p);
    if (e == cudaSuccess) e = launch_pdl(kda_kv_copy_tails_kernel, dim3((unsigned)sms * 4), dim3(256), 0, stream, p);
    return e;
}

cudaError_t launch_kv_truncate(KvCall p, cudaStream_t stream)
{
    static KernelSetup setup;
    const cudaError_t e = setup.get(kda_kv_truncate_kernel, kNt, kMaxMaps, 0, nullptr);
    if (e != cudaSuccess) return e;
    p.lanes = lanes_per_entry(p.B);
    return launch_pdl(kda_kv_truncate_kernel, dim3(entry_ctas(p.B)), dim3(kNt), row_maps_bytes(p, false), stream, p);
}

cudaError_t launch_kv_fork(KvCall p, cudaStream_t stream)
{
    static KernelSetup setup;
    const cudaError_t e = setup.get(kda_kv_fork_kernel, kNt, kMaxMaps, 0, nullptr);
    if (e != cudaSuccess) return e;
    p.lanes = lanes_per_entry(p.B);
    return launch_pdl(kda_kv_fork_kernel, dim3(entry_ctas(p.B)), dim3(kNt), row_maps_bytes(p, true), stream, p);
}

cudaError_t launch_kv_compact(const KvCall &p, cudaStream_t stream)
{
    int sms = 0;
    cudaError_t e = paged_sm_count(&sms);
    if (e == cudaSuccess) e = launch_pdl_cluster(kda_kv_compact_kernel, dim3(kCl), dim3(kNt), 0, kCl, stream, p);
    if (e == cudaSuccess) e = launch_pdl(kda_kv_move_kernel, dim3((unsigned)sms * 8), dim3(256), 0, stream, p);
    return e;
}

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream)
{
    if (p.c.dtype == KDA_T_E4M3) return p.f16 ? append_as<true, true>(p, stream) : append_as<true, false>(p, stream);
    return append_as<false, false>(p, stream);   // a copy of 16-bit words, whatever their type
}

}  // namespace kda
