// kda_kv.cu -- pages of the key-value cache: extend, truncate, fork, compact, append.
//
// The page calls work on small integer arrays (a table row per sequence, a count per page) and
// have to give the same ids whatever order their threads run in.  Ids come from ranks: the r-th
// page asked for gets the r-th free id, both ranks exclusive prefix sums over fixed orders, so no
// result depends on an atomic's order (the atomics add to counts or set flags).
#include <cooperative_groups.h>

#include "kda_paged.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

// One cluster of eight CTAs does the bookkeeping: 8192 threads that can meet at a cluster
// barrier, against one CTA's 1024 (a scan of 64 Ki counts reads 8 per thread instead of 64) and
// against a grid that would need a launch for each phase.
constexpr int kCl = 8, kNt = 1024, kAll = kCl * kNt;

struct ScanMem {
    int warp[32];
    int total;     // this CTA's sum, read by the others through distributed shared memory
};

// Exclusive prefix sum of v over all threads of the cluster in order (CTA rank, thread); every
// thread gets its prefix and the total.  Ends with a barrier, so `sm` can be used again.
__device__ int cluster_scan(cg::cluster_group &cl, ScanMem &sm, int v, int &total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sm.warp[w] = x;
    __syncthreads();
    if (w == 0) {
        int y = sm.warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(~0u, y, o);
            if (lane >= o) y += z;
        }
        sm.warp[lane] = y;
        if (lane == 31) sm.total = y;
    }
    __syncthreads();
    int before = x - v + (w ? sm.warp[w - 1] : 0);
    cl.sync();
    int all = 0;
    const int me = (int)cl.block_rank();
#pragma unroll
    for (int r = 0; r < kCl; r++) {
        const int t = *cl.map_shared_rank(&sm.total, r);
        if (r < me) before += t;
        all += t;
    }
    total = all;
    cl.sync();   // every CTA has read the totals
    return before;
}

struct Scratch {
    int *meta, *mark, *smark, *off, *want, *have, *flag, *cow_src, *cow_dst, *list, *list2;
    __device__ explicit Scratch(const KvCall &p)
    {
        const int R = p.c.rows;
        meta = p.ws;
        mark = p.ws + kKvMeta;
        smark = mark + R;
        off = smark + R;
        want = off + R;
        have = want + R;
        flag = have + R;
        cow_src = flag + R;
        cow_dst = cow_src + R;
        list = cow_dst + R;
        list2 = list + p.c.pages;
    }
};

__device__ __forceinline__ int ceil_pages(const PagedCache &c, int len) { return (int)(((long long)len + c.ps - 1) >> c.ps_log2); }

// The first entry that names each row keeps it: mark[row] = the lowest i with rows[i] = row.
__device__ __forceinline__ void mark_rows(cg::cluster_group &cl, const KvCall &p, const Scratch &s, int g)
{
    for (int i = g; i < p.B; i += kAll)
        if ((unsigned)p.rows[i] < (unsigned)p.c.rows) {
            s.mark[p.rows[i]] = 0x7fffffff;
            s.smark[p.rows[i]] = 0;
        }
    cl.sync();
    for (int i = g; i < p.B; i += kAll)
        if ((unsigned)p.rows[i] < (unsigned)p.c.rows) atomicMin(&s.mark[p.rows[i]], i);
    cl.sync();
}

__device__ __forceinline__ bool owns_row(const KvCall &p, const Scratch &s, int i)
{
    const int r = p.rows[i];
    return (unsigned)r < (unsigned)p.c.rows && __ldcg(&s.mark[r]) == i;
}

__global__ void __launch_bounds__(kNt, 1) kda_kv_extend_kernel(const KvCall p)
{
    __shared__ ScanMem sm;
    cg::cluster_group cl = cg::this_cluster();
    const PagedCache &c = p.c;
    const Scratch s(p);
    const int g = (int)cl.block_rank() * kNt + threadIdx.x;
    grid_dependency_wait();
    if (g == 0) s.meta[0] = 0;   // pages to copy, for the kernel that follows
    mark_rows(cl, p, s, g);
    // what each entry asks for, and its place in the order of the call
    const int per = (p.B + kAll - 1) / kAll;
    int mine = 0;
    for (int i = g * per; i < min(p.B, (g + 1) * per); i++) {
        const int n = p.arg ? p.arg[i] : p.uniform;
        int err = 0, want = 0, copy = 0, have = 0;
        if (!owns_row(p, s, i)) err = KDA_DEVERR_SLOT;
        else if (n < 0) err = KDA_DEVERR_TOKENS;
        else {
            const int r = p.rows[i], len = c.lens[r];
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
    int total = 0, n_free = 0;
    int at = cluster_scan(cl, sm, mine, total);
    for (int i = g * per; i < min(p.B, (g + 1) * per); i++) {
        s.off[i] = at;
        at += s.want[i];
    }
    // the lowest free ids, as many as are asked for
    const int cp = (c.pages + kAll - 1) / kAll, lo = min(c.pages, g * cp), hi = min(c.pages, lo + cp);
    int free_here = 0;
    if (total > 0)
        for (int q = lo; q < hi; q++) free_here += c.refs[q] == 0;
    int rank = cluster_scan(cl, sm, free_here, n_free);
    if (free_here && rank < total)
        for (int q = lo; q < hi; q++)
            if (c.refs[q] == 0) {
                if (rank < total) s.list[rank] = q;
                rank++;
            }
    cl.sync();
    // lengths, and which entries fit
    for (int i = g; i < p.B; i += kAll) {
        const int f = __ldcg(&s.flag[i]), w = __ldcg(&s.want[i]);
        if (f & 4) continue;
        if (w > 0 && __ldcg(&s.off[i]) + (long long)w > n_free) {
            atomicOr(c.err, KDA_DEVERR_NOPAGES);
            s.flag[i] = 4;
            continue;
        }
        const int r = p.rows[i];
        const int n = p.arg ? p.arg[i] : p.uniform;
        if (f & 1) {   // the copy of the shared last page comes first
            int *e = &c.table[(size_t)r * c.width + __ldcg(&s.have[i]) - 1];
            const int from = *e, to = __ldcg(&s.list[__ldcg(&s.off[i])]);
            const int slot = atomicAdd(&s.meta[0], 1);   // any order: the copies are independent
            s.cow_src[slot] = from;
            s.cow_dst[slot] = to;
            s.smark[slot] = c.lens[r] & (c.ps - 1);      // tokens to copy (marks are done with)
            atomicSub(&c.refs[from], 1);
            c.refs[to] = 1;
            *e = to;
        }
        c.lens[r] += n;
    }
    cl.sync();
    // the added pages, one thread each: the entry by bisection over the offsets
    for (int t = g; t < min(total, n_free); t += kAll) {
        int a = 0, b = p.B - 1;   // the last entry whose offset is <= t
        while (a < b) {
            const int m = (a + b + 1) >> 1;
            if (__ldcg(&s.off[m]) <= t) a = m;
            else b = m - 1;
        }
        const int f = __ldcg(&s.flag[a]), j = t - __ldcg(&s.off[a]) - (f & 1);
        if ((f & 4) || j < 0) continue;
        const int page = __ldcg(&s.list[t]);
        c.table[(size_t)p.rows[a] * c.width + __ldcg(&s.have[a]) + j] = page;
        c.refs[page] = 1;
    }
}

// Copies the filled tokens of the shared pages that extend replaced, in every layer: items
// (copy, layer, k or v, head), one warp each, 16 bytes a lane.  Most calls have none, so the grid
// is small and the count is read first.
__global__ void __launch_bounds__(256) kda_kv_copy_tails_kernel(const KvCall p)
{
    const PagedCache &c = p.c;
    const Scratch s(p);
    grid_dependency_wait();
    const int n = s.meta[0];
    const long long items = (long long)n * c.layers * 2 * c.Hkv;
    const int lane = threadIdx.x & 31;
    const size_t row = (size_t)c.D * c.elem(), head = row * c.ps;
    for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (long long)gridDim.x * 8) {
        long long x = it;
        const int h = (int)(x % c.Hkv);
        x /= c.Hkv;
        const int kv = (int)(x & 1);
        x >>= 1;
        const int layer = (int)(x % c.layers), i = (int)(x / c.layers);
        uint8_t *base = (kv ? c.v : c.k) + (size_t)layer * c.pages * c.page_bytes() + h * head;
        const uint4 *src = reinterpret_cast<const uint4 *>(base + (size_t)s.cow_src[i] * c.page_bytes());
        uint4 *dst = reinterpret_cast<uint4 *>(base + (size_t)s.cow_dst[i] * c.page_bytes());
        const int chunks = (int)(s.smark[i] * row / 16);
#pragma unroll 4
        for (int q = lane; q < chunks; q += 32) __stcs(dst + q, __ldcs(src + q));
    }
}

// Threads per entry of a call over n rows: the cluster's threads shared out in powers of two.
__device__ __forceinline__ int lanes_per_entry(int n)
{
    int l = kAll;
    while (l > 32 && (long long)l * n > kAll) l >>= 1;
    return l;
}

__global__ void __launch_bounds__(kNt, 1) kda_kv_truncate_kernel(const KvCall p)
{
    cg::cluster_group cl = cg::this_cluster();
    const PagedCache &c = p.c;
    const Scratch s(p);
    const int g = (int)cl.block_rank() * kNt + threadIdx.x;
    grid_dependency_wait();
    mark_rows(cl, p, s, g);
    const int L = lanes_per_entry(p.B), lane = g & (L - 1);
    for (int i0 = 0; i0 < p.B; i0 += kAll / L) {
        const int i = i0 + g / L;
        bool ok = false;
        int r = 0, keep = 0, have = 0, nl = 0;
        if (i < p.B) {
            int err = 0;
            if (!owns_row(p, s, i)) err = KDA_DEVERR_SLOT;
            else {
                r = p.rows[i];
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
        cl.sync();   // every lane has read its row's length
        if (ok) {
            int *t = c.table + (size_t)r * c.width;
            for (int j = keep + lane; j < have; j += L) {
                const int page = t[j];
                if ((unsigned)page < (unsigned)c.pages) atomicSub(&c.refs[page], 1);
                else atomicOr(c.err, KDA_DEVERR_PAGE);
                t[j] = -1;
            }
            if (lane == 0) c.lens[r] = nl;
        }
    }
}

__global__ void __launch_bounds__(kNt, 1) kda_kv_fork_kernel(const KvCall p)
{
    cg::cluster_group cl = cg::this_cluster();
    const PagedCache &c = p.c;
    const Scratch s(p);
    const int g = (int)cl.block_rank() * kNt + threadIdx.x;
    grid_dependency_wait();
    mark_rows(cl, p, s, g);
    for (int i = g; i < p.B; i += kAll)
        if ((unsigned)p.arg[i] < (unsigned)c.rows) s.smark[p.arg[i]] = 1;
    cl.sync();
    const int L = lanes_per_entry(p.B), lane = g & (L - 1);
    for (int i0 = 0; i0 < p.B; i0 += kAll / L) {
        const int i = i0 + g / L;
        bool ok = false;
        int dst = 0, src = 0, old_pages = 0, new_pages = 0, len = 0;
        if (i < p.B) {
            int err = 0;
            src = p.arg[i];
            if (!owns_row(p, s, i) || (unsigned)src >= (unsigned)c.rows || __ldcg(&s.smark[p.rows[i]])) err = KDA_DEVERR_SLOT;
            else {
                dst = p.rows[i];
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
        cl.sync();   // every lane has read the lengths (a source is never a destination)
        if (ok) {
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
    }
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
    int live = 0, n = 0, moves = 0, holes = 0;
    for (int q = lo; q < hi; q++) live += c.refs[q] != 0;
    cluster_scan(cl, sm, live, n);
    int high = 0, low = 0;
    for (int q = lo; q < hi; q++) {
        const bool used = c.refs[q] != 0;
        high += used && q >= n;
        low += !used && q < n;
    }
    int rh = cluster_scan(cl, sm, high, moves);
    int rl = cluster_scan(cl, sm, low, holes);
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
__device__ __forceinline__ void append_piece(const uint16_t *src, uint8_t *dst, float scale)
{
    const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(src));
    if constexpr (!E4M3) {
        *reinterpret_cast<uint4 *>(dst) = w;
    } else {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float2 f;
            if constexpr (F16) f = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
            else f = make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u));
            // an IEEE division: the code is the rounding of the exact quotient's FP32 value
            f.x = __fdiv_rn(f.x, scale);
            f.y = __fdiv_rn(f.y, scale);
            const __nv_fp8x2_storage_t q = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
            o[i >> 1] |= (uint32_t)q << (16 * (i & 1));
        }
        *reinterpret_cast<uint2 *>(dst) = make_uint2(o[0], o[1]);
    }
}

template <bool E4M3, bool F16>
__global__ void __launch_bounds__(256) kda_kv_append_kernel(const AppendParams p)
{
    const PagedCache &c = p.c;
    const int lane = threadIdx.x & 31;
    const long long tok = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long tokens = p.cu ? p.T : (long long)p.B * p.T;
    grid_dependency_wait();
    if (tok >= tokens) return;
    int b, t, n;
    long long koff, voff;
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
        koff = tok * p.kl.token;
        voff = tok * p.vl.token;
    } else {
        b = (int)(tok / p.T);
        t = (int)(tok - (long long)b * p.T);
        n = p.n_tokens ? p.n_tokens[b] : p.T;
        koff = b * p.kl.seq + t * p.kl.token;
        voff = b * p.vl.seq + t * p.vl.token;
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
    const int per_log2 = c.D == 128 ? 4 : 3, pieces = c.Hkv << per_log2;   // 8 elements each
#pragma unroll 4
    for (int q = lane; q < pieces; q += 32) {
        const int h = q >> per_log2, i = q & ((1 << per_log2) - 1);
        const size_t to = at + h * head + (size_t)i * 8 * ES;
        append_piece<E4M3, F16>(p.k + koff + h * p.kl.head + i * 8, c.k + to, E4M3 ? c.k_scale[p.layer * c.Hkv + h] : 1.f);
        append_piece<E4M3, F16>(p.v + voff + h * p.vl.head + i * 8, c.v + to, E4M3 ? c.v_scale[p.layer * c.Hkv + h] : 1.f);
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
    int sms = 0;
    cudaError_t e = paged_sm_count(&sms);
    if (e == cudaSuccess) e = launch_pdl_cluster(kda_kv_extend_kernel, dim3(kCl), dim3(kNt), kCl, stream, p);
    if (e == cudaSuccess) e = launch_pdl(kda_kv_copy_tails_kernel, dim3((unsigned)sms), dim3(256), 0, stream, p);
    return e;
}

cudaError_t launch_kv_truncate(const KvCall &p, cudaStream_t stream)
{
    return launch_pdl_cluster(kda_kv_truncate_kernel, dim3(kCl), dim3(kNt), kCl, stream, p);
}

cudaError_t launch_kv_fork(const KvCall &p, cudaStream_t stream)
{
    return launch_pdl_cluster(kda_kv_fork_kernel, dim3(kCl), dim3(kNt), kCl, stream, p);
}

cudaError_t launch_kv_compact(const KvCall &p, cudaStream_t stream)
{
    int sms = 0;
    cudaError_t e = paged_sm_count(&sms);
    if (e == cudaSuccess) e = launch_pdl_cluster(kda_kv_compact_kernel, dim3(kCl), dim3(kNt), kCl, stream, p);
    if (e == cudaSuccess) e = launch_pdl(kda_kv_move_kernel, dim3((unsigned)sms * 8), dim3(256), 0, stream, p);
    return e;
}

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream)
{
    if (p.c.dtype == KDA_T_E4M3) return p.f16 ? append_as<true, true>(p, stream) : append_as<true, false>(p, stream);
    return append_as<false, false>(p, stream);   // a copy of 16-bit words, whatever their type
}

}  // namespace kda
