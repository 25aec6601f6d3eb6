// kda_attn_decode.cuh -- attention of a few new tokens per sequence over a paged key-value cache
// (kda_attn_decode): decode, draft verify and mixed steps.
//
// Mathematics.  For one sequence and key head the rows are the call's (token, query head) pairs,
// R = n * G of them; per block of keys S^T = K Q^T, P = exp2(S^T - m) with a running maximum m and
// sum l per row, O^T += V^T P^T, both products on mma.sync m16n8k16 with keys (or head dims) as the
// 16 rows and 8 query rows as columns.  Keys and head dims are summed over, so their order within a
// block is free: each thread takes 16 contiguous bytes of a key as its A fragments for two k-steps
// and takes the same elements of q, and V's fragments pair the same element of two keys (one byte
// permutation a word).  P^T becomes the B operand by transposing 8x8 matrices between lanes.
//
// Bound.  Every key and value byte is used for R rows only: HBM bound (R <= 32 needs at most 1/8 of
// the tensor rate).  So the design is about bytes in flight and an even split.  Each warp owns a ring
// of cp.async stages (16 keys and values a stage; two to four stages, 12 to 24 KiB a warp, 8 to 16 warps and
// 144 to 192 KiB an SM, see Cfg, against about 45 KiB that the latency-bandwidth product asks of an SM; with 4 bits 32 keys and
// values a stage, three to six stages, 11 to 23 KiB a warp and 162 to 216 KiB an SM), with no
// CTA barrier inside a run of keys.  All tiles of all (sequence, key head, row block) units are laid out in one line and
// cut into equal runs, one per CTA, so ragged lengths load the SMs evenly; a unit that spans several
// CTAs leaves partial (m, l, O) in the workspace and the CTA that finishes last joins them in the
// fixed order of the pieces.  No result depends on which CTA that is.
//
// Rows of a page that no token sees are not read: cp.async writes zeros for them, so whatever the
// page holds there (NaN included) cannot reach the products.
//
// 4-bit caches (E2M1 codes, an E4M3 scale for each 16 elements of a key): bytes halve again and the instructions do not.  Two codes a
// conversion and a product with their scale, both exact in halves, are 256 of about 630 instructions for 32 keys of 128 dims and a
// block of 8 rows; in long runs HBM bounds it all the same (608 sequences of 32768 tokens: 5.8 TB/s), in short units their
// starts and merges do (256 sequences of 1 to 4096 tokens, 8 heads: 120 us, 4.4 TB/s).  With more rows latencies do, at 8 to 12 warps an
// SM: 64 x 4096 tokens, 20 rows 119 us, 32 rows 149 (issue slots 40 % busy; these blocks spill 84 bytes of loads a thread, with half
// queries 252: 178 us; of 64 dims 100 and 28: 95 and 91 us).
#pragma once

#include "kda_attn_common.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kStep = 16;                 // keys of a product
constexpr int kMaxCtas = 1024;            // bound of the grid, sizes the workspace
constexpr int kUnitRows = 32;
// A unit counts for this many tiles more than it has: starting one (queries, page ids, the first keys,
// the merge) takes as long as some tiles.  Without it a run of one-tile units held the call up: 64 ragged
// sequences, four drafts, 1024 window: 70 us, with 2 / 4 / 8: 47 / 41 / 41 us; 131072 tokens of one
// sequence: 91 us, 90 / 89 / 94 us.
constexpr int kUnitCost = 4;
// How many places longer a run may get for whole units to each CTA (see where the runs are made): Cfg::UNEVEN, or kUnevenShort
// where the runs are shorter than a unit's start.  A place is a tile, 64 keys of a 16-bit or E4M3 cache and 128 of a 4-bit one.
// 16 bits and E4M3, 12 and 8: measured both ways on 44 forms (64 and 128 dims, 1 to 100 sequences of 300 to 2048 tokens, 32
// query and 8 key heads, one and four tokens): the 22 that get whole units gain 1 to 38 % by them, but for two that lose
// 1.5 %; of the 22 that are cut, whole units would cost 17 forms 1 to 23 % (one sequence of 517 tokens, 12 places more: 8.5
// us cut, 10.2 whole; of 300 tokens, 8 more: 9.2 and 7.7) and would gain five of 64 dims 2 to 16 %.  64 ragged sequences in a
// 1024 window, 20 rows a unit: 35.3 us with cut units, 31.1 with whole ones (9 more).
// 4 bits, 7 and 8: measured both ways on 208 forms (64 and 128 dims, 1 to 152 sequences of 300 to 8192 tokens, windows of 512 to
// 2048, 8 key heads, 4 to 32 rows).  Longer runs: whole units of 1 to 7 places more take 1 to 43 % less time than cut ones, of 8
// and 9 from 9 % less to 20 % more, of 10 and above 4 to 48 % more (64 sequences of 1024 tokens, 16 rows, 10 more: 40.3 us cut,
// 45.2 whole; but three units of 15 places for a run of 37: 83 us cut, 77 whole).  Short runs: of 8 at most from 37 % less (four
// sequences of 517 tokens, 32 rows: 32.6 us cut, 20.5 whole) to 15 % more, of 9 and above from 12 % less to 131 % more.
constexpr int kUnevenShort = 8;

template <typename T>
__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    if constexpr (T::is_half)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ... of halves, from zero
__device__ __forceinline__ void mma16816_zero(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Transposes an 8x8 matrix of 16-bit elements held one row per quad.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

template <int D, int KV, int NB>
struct Cfg {
    static constexpr int RB = KV == kKv16 ? D * 2 : KV == kKvE4M3 ? D : D / 2;   // bytes of a key (its codes)
    static constexpr int SB = KV == kKvE2M1 ? D / 16 : 0; // ... and of its block scales
    static constexpr int CH = RB / 16;                    // 16-byte chunks of a key
    // Keys of a warp's step.  Two groups of 16 with 4 bits: their page ids, addresses, bounds and maximum took as many
    // instructions as a third of their arithmetic.  256 sequences of 1 to 4096 tokens, 8 heads: 139 us with 16 keys, 120 with
    // 32 (and addresses kept from step to step); in long runs 5.8 TB/s.
    static constexpr int KEYS = KV == kKvE2M1 ? 2 * kStep : kStep, TILE = kWarps * KEYS;   // ... and of a tile: a step of each warp
    static constexpr int STAGE = 2 * KEYS * (RB + SB);    // keys, values, then both's block scales
    static constexpr int V_AT = KEYS * RB, KS_AT = 2 * V_AT, VS_AT = KS_AT + KEYS * SB;
    // CTAs of an SM: as many as the accumulators (D NB / 4 registers) leave room for.  A warp's step is a
    // chain of latencies (scores, exponentials, product), which other warps cover: two CTAs everywhere
    // against this, 64 x 4096 tokens, 8 heads, E4M3: 153 us, 129 us; bfloat16 (HBM bound) 171 us both.
    // 4-bit blocks of 24 rows one fewer: with more they spill (20 rows, 64 x 4096 tokens, 8 heads: 131 us, 122 of 128 dims, 84 and 76
    // of 64; in a 1024 window, a unit a CTA, 30.2 and 31.2).
    static constexpr int OCC = D * NB >= 512 ? 2 : KV == kKvE2M1 && NB == 3 ? (D == 64 ? 3 : 2) : (RB == 256 || D * NB >= 256) ? 3 : 4;
    static constexpr bool Q_SMEM = NB > 1;                // queries in shared memory instead of registers
    static constexpr int Q_BYTES = Q_SMEM ? NB * 8 * D * 2 : 0;
    // Sequences whose (row, length, tokens) are kept on chip.  E2M1: three stages and four CTAs take all of the 228 KB but 2 KB a CTA.
    static constexpr int SEQS = KV == kKvE2M1 ? 224 : 256;
    static constexpr int NS_FIT = KV == kKvE2M1 ? (228 * 1024 / OCC - 1024 - 8 * SEQS - 128 - Q_BYTES) / (kWarps * STAGE)
                                                : (220 * 1024 / OCC - 2048 - Q_BYTES) / (kWarps * STAGE);
    static constexpr int NS = NS_FIT > 6 ? 6 : NS_FIT;    // stages of a warp's ring
    static constexpr int RING = kWarps * NS * STAGE;
    // the pieces of a unit are merged in the ring's place
    static constexpr int MERGE = kWarps * 8 * NB * (D + 2) * 4;
    static constexpr int SMEM = (RING > MERGE ? RING : MERGE) + Q_BYTES;
    // chunk c of row r is stored at chunk c ^ swz(r): conflict-free for the fragment loads
    // (K: eight lanes read four chunks of two rows; V: two chunks of four even rows)
    static __device__ __forceinline__ int swz_k(int r) { return CH >= 8 ? 4 * (r & 1) : 0; }
    static __device__ __forceinline__ int swz_v(int r) { return KV == kKvE2M1 ? 0 : CH >= 8 ? 2 * ((r >> 1) & 3) : (r >> 1) & 3; }
    // where chunk c of value row r of an E2M1 step is stored: its rows are shorter than the banks are wide, so the
    // chunks of the 128 bytes that hold 2 (or 4) rows change places (lanes read 8, or 4, bytes of every second row)
    static __device__ __forceinline__ int v_at(int r, int c)
    {
        return D == 128 ? (r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (2 * ((r >> 1) & 3))) * 16)
                        : (r >> 2) * 128 + ((((r & 3) * 2 + c) ^ (2 * ((r >> 2) & 1))) * 16);
    }
    static constexpr int UNEVEN = KV == kKvE2M1 ? 7 : 12;   // see kUnevenShort
    // head dim of the first of the two elements that accumulator block m of lane group g holds
    static __device__ __forceinline__ int dim(int m, int g) { return KV != kKv16 ? (D / 8) * g + 2 * m : 64 * (m >> 2) + 8 * g + 2 * (m & 3); }
};

struct Partials {   // workspace: counters, then for each CTA two slots of (m, l, O)
    int *count, *group;   // [kMaxCtas] of units by first CTA, [2 kMaxCtas] of groups by first slot
    float *data;
    static constexpr size_t kCounters = kAttnCounters;
    static_assert(kCounters >= 3 * kMaxCtas, "units and groups");
    static constexpr size_t slot_floats(int D) { return (size_t)kUnitRows * (D + 2); }
    __device__ float *slot(int s, int D) const { return data + (size_t)s * slot_floats(D); }
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp16(uint32_t dst, const uint8_t *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const uint8_t *src, bool read)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}

// Runs of tiles are counted in 64 bits (rows that share pages can hold more keys than memory); the
// divisions take the 32-bit path whenever the numbers allow it.
__device__ __forceinline__ long long div_pos(long long a, long long b)
{
    return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

template <int D, typename Q, int KV, int NB>
__global__ void __launch_bounds__(kThreads, Cfg<D, KV, NB>::OCC) kda_attn_decode_kernel(const AttnParams p)
{
    using C = Cfg<D, KV, NB>;
    constexpr bool CODES = KV != kKv16;
    // type of both products: E4M3 codes are exact halves, and so are E2M1 codes times their E4M3 scale (two bits by
    // four, 2^-10 to 2688)
    using P = std::conditional_t<CODES, Half, Q>;
    constexpr int kSeqs = C::SEQS;
    constexpr int MT = D / 16;                    // accumulator blocks (16 head dims)
    constexpr int ROWS = 8 * NB;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long sh_prefix, sh_warp[kWarps];
    __shared__ int sh_b, sh_last, sh_units[kWarps], sh_most[kWarps], sh_seq[2][kSeqs];   // row and tokens, length
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, cc = lane & 3;
    const int W = p.window > 0 ? p.window : 0x7fffffff, S = p.window > 0 ? p.sinks : 0;
    Partials part;
    part.count = reinterpret_cast<int *>(p.ws);
    part.group = part.count + kMaxCtas;
    part.data = reinterpret_cast<float *>(p.ws + Partials::kCounters * sizeof(int));

    grid_dependency_wait();

    // ---- this CTA's run of tiles
    auto load_seq = [&](int b, bool report) { return seq_info(c, p.rows[b], p.n_tokens ? p.n_tokens[b] : p.T, p.T, report); };
    int place = 0;   // places of a unit on the line of work: kUnitCost, then one for each of its tiles, or (not 0) this many
    auto tiles_of = [&](const SeqInfo &s, int &kt, int &mt) -> long long {   // kt tiles in each of Hkv * mt units
        kt = mt = 0;
        if (!s.ok || s.n == 0) return 0;
        const KeyRange<C::TILE> r(s.len - s.n, s.len - 1, s.len, W, S);
        kt = max(1, r.count);
        mt = (s.n * p.G + ROWS - 1) / ROWS;
        return (long long)(place ? place : kt + kUnitCost) * mt * c.Hkv;
    };
    const int per = (p.B + kThreads - 1) / kThreads, b_lo = min(p.B, tid * per), b_hi = min(p.B, b_lo + per);
    long long mine = 0;
    int kt, mt, units = 0, most = 0;   // (units: 2^20 at most)
    for (int b = b_lo; b < b_hi; b++) {
        const SeqInfo s = load_seq(b, blockIdx.x == 0);
        if (b < kSeqs) sh_seq[0][b] = (s.row & (kMaxRows - 1)) | (s.ok ? s.n : 0) * kMaxRows, sh_seq[1][b] = s.len;
        mine += tiles_of(s, kt, mt);
        units = min(units + mt * c.Hkv, 1 << 20);
        if (mt) most = max(most, kt + kUnitCost);
    }
    auto seq_of = [&](int b) {   // after the barrier below
        if (b >= kSeqs) return load_seq(b, false);
        SeqInfo s;
        s.row = sh_seq[0][b] & (kMaxRows - 1), s.len = sh_seq[1][b], s.n = sh_seq[0][b] / kMaxRows, s.ok = true;
        return s;
    };
    long long before = mine;
    const int warp_units = __reduce_add_sync(~0u, units);
    most = __reduce_max_sync(~0u, most);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) sh_warp[w] = before, sh_units[w] = warp_units, sh_most[w] = most;
    __syncthreads();
    before -= mine;
    long long total = 0;
    int all_units = 0;
#pragma unroll
    for (int i = 0; i < kWarps; i++) {
        if (i < w) before += sh_warp[i];
        total += sh_warp[i];
        all_units += sh_units[i];
        most = max(most, sh_most[i]);
    }
    long long chunk = max(1ll, div_pos(total + gridDim.x - 1, gridDim.x));
    // Whole units to each CTA, places as many as the longest unit has, where the longest run gets no more than C::UNEVEN
    // places longer (kUnevenShort, where the runs are shorter than a unit's start): no unit is started twice and none
    // is joined.
    const int each = all_units <= (int)gridDim.x ? 1 : (all_units + gridDim.x - 1) / gridDim.x;
    if (all_units < 1 << 20 && (long long)each * most <= chunk + (chunk > kUnitCost ? C::UNEVEN : kUnevenShort)) {
        int x = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        x -= units;
#pragma unroll
        for (int i = 0; i < kWarps; i++)
            if (i < w) x += sh_units[i];
        place = most;
        mine = (long long)units * most;
        before = (long long)x * most;
        total = (long long)all_units * most;
        chunk = max(1ll, (long long)each * most);
    }
    const long long begin = blockIdx.x * chunk, end = min(total, begin + chunk);
    if (begin >= end) return;
    if (begin >= before && begin < before + mine) {
        long long at = before;
        for (int b = b_lo; b < b_hi; b++) {
            const long long n = tiles_of(seq_of(b), kt, mt);
            if (begin < at + n) {
                sh_b = b;
                sh_prefix = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    int b = sh_b;
    long long prefix = sh_prefix;
    SeqInfo seq = seq_of(b);
    long long seq_tiles = tiles_of(seq, kt, mt);

    uint2 *q_sm = reinterpret_cast<uint2 *>(smem);        // queries, [NB][D / 16][32 lanes]
    uint8_t *ring_p = smem + C::Q_BYTES + w * (C::NS * C::STAGE);
    const uint32_t ring = smem_u32(ring_p), q_at = smem_u32(smem) + lane * 8;
    float *mg = reinterpret_cast<float *>(smem + C::Q_BYTES);          // merge buffer: O [warp][ROWS][D], m, l [warp][ROWS]
    float *mg_m = mg + kWarps * ROWS * D, *mg_l = mg_m + kWarps * ROWS;

    int pages_of = -1, first_now = -1, first_next = -1;   // whose pages of tiles 0 to 63 this lane holds
    [[maybe_unused]] int first_now2 = -1, first_next2 = -1;
    long long at = begin;
    while (at < end) {
        while (at >= prefix + seq_tiles) {   // next sequence with work (there is one: at < total)
            prefix += seq_tiles;
            seq = seq_of(++b);
            seq_tiles = tiles_of(seq, kt, mt);
        }
        const int unit = place ? place : kt + kUnitCost, local = (int)div_pos(at - prefix, unit);
        const int h = local / mt, mb = local % mt;
        const long long u0 = prefix + (long long)local * unit + unit - kt;   // the unit's tiles: places [u0, u0 + kt)
        if (u0 >= end) break;   // they belong to the next CTAs
        const int ta = (int)(max(at, u0) - u0), tb = (int)min((long long)kt, end - u0);
        const int n_rows = min(ROWS, seq.n * p.G - mb * ROWS);
        const int p0 = seq.len - seq.n;
        const KeyRange<C::TILE> kr(p0, seq.len - 1, seq.len, W, S);
        const int lo_all = (int)max(0ll, (long long)seq.len - W);         // every token sees [lo_all, p0]
        const uint32_t page_bytes = (uint32_t)c.page_bytes();   // under 2^27
        const uint8_t *k_head = c.k + ((size_t)p.layer * c.pages * c.Hkv + h) * ((size_t)c.ps * (C::RB + C::SB)), *k_base = k_head + lane * 16;
        const ptrdiff_t v_minus_k = c.v - c.k;
        // E2M1: lanes copy 16 bytes of a step's block scales, the first half of them keys', the others values'; with pages of
        // 16 tokens a step has two pages, whose halves of the scales are each other lanes'
        constexpr int SC = 2 * C::KEYS * C::SB / 16;
        const bool two_pages = KV == kKvE2M1 && c.ps < C::KEYS, second = two_pages && lane % max(1, SC / 2) >= SC / 4;
        const uint8_t *sc_base = KV == kKvE2M1 ? k_head + (lane < SC / 2 ? 0 : v_minus_k) + (size_t)c.ps * C::RB + lane % max(1, SC / (two_pages ? 4 : 2)) * 16 : nullptr;
        // where a lane's pieces go: the swizzles of a step's rows differ from its first row's by constants
        const uint32_t dst_k = (lane / C::CH) * C::RB + (((lane % C::CH) ^ C::swz_k(lane / C::CH)) * 16);
        const uint32_t dst_v = KV == kKvE2M1 ? C::v_at(lane / C::CH, lane % C::CH)
                                             : (lane / C::CH) * C::RB + (((lane % C::CH) ^ C::swz_v(lane / C::CH)) * 16);

        // queries: rows nb * 8 + g, the elements this thread multiplies
        uint32_t qf[C::Q_SMEM ? 1 : D / 16][2];
        float sc[NB][2];      // scale of rows 2 cc, 2 cc + 1, in log2 units
        int row_pos[NB][2];   // and their tokens' positions
        const float sc_head = p.scale_log2 * (CODES ? c.k_scale[p.layer * c.Hkv + h] : 1.f);
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
            const int r = nb * 8 + g;
            const int t = (mb * ROWS + r) / p.G, hq = h * p.G + (mb * ROWS + r) - t * p.G;
            const uint16_t *src = p.q + b * p.ql.seq + t * p.ql.token + hq * p.ql.head;
            uint4 x[D / 32];
#pragma unroll
            for (int j = 0; j < D / 32; j++) {
                // 16-bit cache: chunk cc + 4 j of 8 elements; E4M3: 16-element chunks, this is half (j & 1) of chunk cc + 4 (j / 2);
                // E2M1: a quarter of the key
                const int e = KV == kKv16 ? 8 * (cc + 4 * j) : KV == kKvE4M3 ? 16 * (cc + 4 * (j >> 1)) + 8 * (j & 1) : (D / 4) * cc + 8 * j;
                x[j] = r < n_rows ? __ldg(reinterpret_cast<const uint4 *>(src + e)) : make_uint4(0, 0, 0, 0);
            }
            float up = 1.f;
            if constexpr (CODES && !Q::is_half) {
                uint32_t mag = 0;
#pragma unroll
                for (int j = 0; j < D / 32; j++) mag = max_magnitude(mag, x[j]);
                mag = max(mag, __shfl_xor_sync(~0u, mag, 1));
                mag = max(mag, __shfl_xor_sync(~0u, mag, 2));
                float down;
                query_scale(mag, down, up);
#pragma unroll
                for (int j = 0; j < D / 32; j++) x[j] = scaled_halves(x[j], down);
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                sc[nb][i] = score_scale(sc_head * (CODES && !Q::is_half ? __shfl_sync(~0u, up, 4 * (2 * cc + i)) : 1.f));
                row_pos[nb][i] = p0 + (mb * ROWS + nb * 8 + 2 * cc + i) / p.G;
            }
#pragma unroll
            for (int j = 0; j < D / 32; j++) {
                if constexpr (C::Q_SMEM) {
                    if (w == (nb & 3)) {
                        q_sm[(nb * (D / 16) + 2 * j) * 32 + lane] = make_uint2(x[j].x, x[j].y);
                        q_sm[(nb * (D / 16) + 2 * j + 1) * 32 + lane] = make_uint2(x[j].z, x[j].w);
                    }
                } else {
                    qf[2 * j][0] = x[j].x, qf[2 * j][1] = x[j].y;
                    qf[2 * j + 1][0] = x[j].z, qf[2 * j + 1][1] = x[j].w;
                }
            }
        }
        if constexpr (C::Q_SMEM) __syncthreads();

        float acc[MT][NB][4];
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int i = 0; i < 4; i++) acc[m][nb][i] = 0.f;
        float row_m[NB][2], row_l[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; nb++) row_m[nb][0] = row_m[nb][1] = -INFINITY, row_l[nb][0] = row_l[nb][1] = 0.f;

        // page ids of this warp's next 32 steps, one per lane, and of the 32 after them
        // (E2M1: `sub` is the step's second group of 16 keys; its page is another one where pages have 16 tokens)
        auto key_of = [&](int t) { return kr.tile(t) * C::TILE + w * C::KEYS; };
        auto step_used = [&](int k0) { return k0 < kr.end && (k0 + kStep > kr.lo || k0 < S); };
        [[maybe_unused]] auto step4_used = [&](int k0) { return k0 < kr.end && (k0 + C::KEYS > kr.lo || k0 < S); };
        auto load_pages = [&](int t0, int sub) {
            const int t = t0 + lane;
            if (t >= kt) return -1;
            const int k0 = key_of(t) + sub * kStep;
            const bool used = KV != kKvE2M1 || two_pages ? step_used(k0) : sub == 0 && step4_used(k0);
            return used ? __ldg(c.table + (size_t)seq.row * c.width + (k0 >> c.ps_log2)) : -1;
        };
        // a sequence's next unit (another head, the same pages) begins with those of its last one
        int pages_at = ta, pages_now, pages_next;
        [[maybe_unused]] int pages_now2, pages_next2;
        if (ta == 0 && pages_of == b) {
            pages_now = first_now, pages_next = first_next;
            if constexpr (KV == kKvE2M1) pages_now2 = first_now2, pages_next2 = first_next2;
        } else {
            pages_now = load_pages(ta, 0);
            pages_next = load_pages(ta + 32, 0);
            if constexpr (KV == kKvE2M1) pages_now2 = load_pages(ta, 1), pages_next2 = load_pages(ta + 32, 1);
            if (ta == 0) {
                pages_of = b, first_now = pages_now, first_next = pages_next;
                if constexpr (KV == kKvE2M1) first_now2 = pages_now2, first_next2 = pages_next2;
            }
        }

        uint32_t bad = 0;   // bit s: the step in stage s has no page; E2M1: two bits, for its groups
        [[maybe_unused]] auto issue4 = [&](int k0, int page, int page2, int stage) {
            const uint32_t to = ring + stage * C::STAGE, in = k0 & (c.ps - 1);
            constexpr int HALF = kStep * C::RB;
            if (k0 + C::KEYS <= kr.end && (k0 >= kr.lo || k0 + C::KEYS <= S) && (unsigned)page < (unsigned)c.pages && (unsigned)page2 < (unsigned)c.pages) {
                // some token sees every key, and all have a page
                if (bad) bad &= ~(3u << 2 * stage);
                const uint8_t *s1 = k_base + (size_t)(uint32_t)page * page_bytes + in * C::RB, *s2 = s1 + v_minus_k;
                const uint32_t dk = to + lane * 16, dv = to + C::V_AT + dst_v;
#pragma unroll
                for (int i = 0; i < HALF; i += 512) cp16(dk + i, s1 + i), cp16(dv + i, s2 + i);
                if (two_pages) {
                    const uint8_t *s3 = k_base + (size_t)(uint32_t)page2 * page_bytes, *s4 = s3 + v_minus_k;
#pragma unroll
                    for (int i = 0; i < HALF; i += 512) cp16(dk + HALF + i, s3 + i), cp16(dv + HALF + i, s4 + i);
                } else {
#pragma unroll
                    for (int i = HALF; i < 2 * HALF; i += 512) cp16(dk + i, s1 + i), cp16(dv + i, s2 + i);
                }
                if (SC == 32 || lane < SC) cp16(dk + C::KS_AT, sc_base + (size_t)(uint32_t)(second ? page2 : page) * page_bytes + in * C::SB);
                return;
            }
            if (!step4_used(k0)) return;
            for (int sub = 0; sub < 2; sub++) {   // zeros for the keys that no token sees, or that have no page
                const int g0 = k0 + sub * kStep, pg = sub ? page2 : page;
                // (a step's two groups are in one page where pages have more than 16 tokens, whichever of them is seen)
                const bool used = step_used(g0), ok = used && (unsigned)pg < (unsigned)c.pages;
                bad = used && !ok ? bad | (1u << (2 * stage + sub)) : bad & ~(1u << (2 * stage + sub));
                if (used && !ok && lane == 0) atomicOr(c.err, KDA_DEVERR_PAGE);
                const uint8_t *head = k_head + (ok ? (size_t)(uint32_t)pg * page_bytes : 0);
                const int row0 = g0 & (c.ps - 1);
                constexpr int PER = 32 / C::CH;
#pragma unroll
                for (int i = 0; i < kStep / PER; i++) {
                    const int r = i * PER + lane / C::CH, j = g0 + r;
                    const bool read = ok && j < kr.end && (j >= kr.lo || j < S);
                    const uint8_t *src = head + (row0 + r) * C::RB + lane % C::CH * 16;
                    const uint32_t dst = to + sub * kStep * C::RB;
                    cp16_or_zero(dst + lane * 16 + i * 512, src, read);
                    cp16_or_zero(dst + C::V_AT + dst_v + i * 512, src + v_minus_k, read);
                }
                const int r = lane % kStep, j = g0 + r;   // block scales: half the lanes keys', the others values'
                cp_async_small<C::SB>(to + (lane < kStep ? C::KS_AT : C::VS_AT) + (sub * kStep + r) * C::SB,
                                      head + (lane < kStep ? 0 : v_minus_k) + (size_t)c.ps * C::RB + (row0 + r) * C::SB,
                                      ok && j < kr.end && (j >= kr.lo || j < S) ? C::SB : 0);
            }
        };
        auto issue = [&](int t, int stage) {
            if (t < tb) {
                if (t - pages_at >= 32) {
                    pages_at += 32;
                    pages_now = pages_next;
                    pages_next = load_pages(pages_at + 32, 0);
                    if constexpr (KV == kKvE2M1) pages_now2 = pages_next2, pages_next2 = load_pages(pages_at + 32, 1);
                }
                const int k0 = key_of(t);
                const int page = __shfl_sync(~0u, pages_now, t - pages_at);
                if constexpr (KV == kKvE2M1) {
                    issue4(k0, page, two_pages ? __shfl_sync(~0u, pages_now2, t - pages_at) : page, stage);
                    cp_async_commit();
                    return;
                }
                if (step_used(k0)) {
                    const bool ok = (unsigned)page < (unsigned)c.pages;
                    bad = ok ? bad & ~(1u << stage) : bad | (1u << stage);
                    if (!ok) {
                        if (lane == 0) atomicOr(c.err, KDA_DEVERR_PAGE);
                    } else {
                        // this lane's pieces: 16 bytes of row r0 + i * 32 / CH, all 512 bytes apart
                        const uint8_t *sk = k_base + (size_t)(uint32_t)page * page_bytes + (k0 & (c.ps - 1)) * C::RB, *sv = sk + v_minus_k;
                        const uint32_t dk = ring + stage * C::STAGE + dst_k, dv = ring + stage * C::STAGE + kStep * C::RB;
                        constexpr int PER = 32 / C::CH;   // rows of a piece's step
                        if (k0 + kStep <= kr.end && (k0 >= kr.lo || k0 + kStep <= S)) {
#pragma unroll
                            for (int i = 0; i < kStep / PER; i++) {
                                cp16(dk + i * 512, sk + i * 512);
                                cp16(dv + i * 512 + (dst_v ^ (C::swz_v(i * PER) * 16)), sv + i * 512);
                            }
                        } else {   // zeros for the keys that no token sees
#pragma unroll
                            for (int i = 0; i < kStep / PER; i++) {
                                const int j = k0 + i * PER + lane / C::CH;
                                const bool read = j < kr.end && (j >= kr.lo || j < S);
                                cp16_or_zero(dk + i * 512, sk + i * 512, read);
                                cp16_or_zero(dv + i * 512 + (dst_v ^ (C::swz_v(i * PER) * 16)), sv + i * 512, read);
                            }
                        }
                    }
                }
            }
            cp_async_commit();
        };

        // A step of 32 4-bit keys: the scores of both groups, one look at the maximum, both groups' values.
        float row_b[NB][2] = {};   // row_m, but 0 while a row has seen no key
        // Where this lane's values and their block scales are in a stage: row 2 cc; row 2 cc + 1 is in the neighbouring chunks, D / 2
        // bytes away (stages begin at multiples of 128 bytes).
        const uint32_t vo = KV != kKvE2M1 ? 0 : C::V_AT + C::v_at(2 * cc, D == 128 ? g >> 1 : g >> 2) + (D == 128 ? 8 * (g & 1) : 4 * (g & 3));
        const uint32_t vso = C::VS_AT + 2 * cc * C::SB + (D == 128 ? g : g >> 1);
        static_assert(KV != kKvE2M1 || C::STAGE % 128 == 0, "");
        [[maybe_unused]] auto step4 = [&](int k0, int stage) {
            const uint32_t at = ring + stage * C::STAGE, at_k = at + lane * (D / 8), at_ks = at + lane * (D / 64), at_v = at + vo, at_v1 = at_v ^ (D / 2), at_vs = at + vso;
            float s[2][NB][4];
#pragma unroll
            for (int sub = 0; sub < 2; sub++) {
                // a quarter of the key for each lane, one or two blocks of 16 elements
                constexpr int NW = D / 32;
                uint32_t xs[NW], ys[NW], sx[2], sy[2];
                const uint32_t kb = at_k + sub * kStep * C::RB, ks = at_ks + C::KS_AT + sub * kStep * C::SB;
                if constexpr (D == 128) {
                    const uint4 x = lds128(kb), y = lds128(kb + 8 * C::RB);
                    xs[0] = x.x, xs[1] = x.y, xs[2] = x.z, xs[3] = x.w;
                    ys[0] = y.x, ys[1] = y.y, ys[2] = y.z, ys[3] = y.w;
                    const uint32_t a = e4m3x2_half2(lds_u16(ks)), b = e4m3x2_half2(lds_u16(ks + 8 * C::SB));
                    sx[0] = __byte_perm(a, a, 0x1010), sx[1] = __byte_perm(a, a, 0x3232);
                    sy[0] = __byte_perm(b, b, 0x1010), sy[1] = __byte_perm(b, b, 0x3232);
                } else {
                    const uint2 x = lds64(kb), y = lds64(kb + 8 * C::RB);
                    xs[0] = x.x, xs[1] = x.y, ys[0] = y.x, ys[1] = y.y;
                    sx[0] = e4m3x2_half2(lds_u8(ks) * 0x101u), sy[0] = e4m3x2_half2(lds_u8(ks + 8 * C::SB) * 0x101u);
                }
#pragma unroll
                for (int u = 0; u < NW; u++) {
                    uint32_t x[4], y[4];
                    e2m1x8_half8(xs[u], x);
                    e2m1x8_half8(ys[u], y);
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const uint32_t a[4] = {hmul2(x[2 * i], sx[u / 2]), hmul2(y[2 * i], sy[u / 2]), hmul2(x[2 * i + 1], sx[u / 2]), hmul2(y[2 * i + 1], sy[u / 2])};
#pragma unroll
                        for (int nb = 0; nb < NB; nb++) {
                            uint2 q;
                            if constexpr (C::Q_SMEM) q = lds64(q_at + (nb * (D / 16) + 2 * u + i) * 256);
                            else q = make_uint2(qf[2 * u + i][0], qf[2 * u + i][1]);
                            if (u == 0 && i == 0) mma16816_zero(s[sub][nb], a, q.x, q.y);
                            else mma16816<P>(s[sub][nb], a, q.x, q.y);
                        }
                    }
                }
            }
            // s[sub][nb]: keys k0 + 16 sub + g (+ 8), rows nb * 8 + 2 cc (+ 1); in units of log2
            if (!(k0 + C::KEYS - 1 <= p0 && (k0 >= lo_all || k0 + C::KEYS <= S) && bad == 0)) {
#pragma unroll
                for (int sub = 0; sub < 2; sub++)
#pragma unroll
                    for (int nb = 0; nb < NB; nb++)
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            if ((bad >> (2 * stage + sub) & 1) || !key_visible(k0 + sub * kStep + g + 8 * (i >> 1), row_pos[nb][i & 1], W, S)) s[sub][nb][i] = -INFINITY;
            }
            bool grown = false;
            float top[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    top[nb][i] = fmaxf(fmaxf(s[0][nb][i], s[0][nb][i + 2]), fmaxf(s[1][nb][i], s[1][nb][i + 2])) * sc[nb][i];
                    grown |= top[nb][i] > row_m[nb][i] + (P::kShift + P::kGrow);
                }
            if (__any_sync(~0u, grown)) {
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        float mx = top[nb][i];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
                        const float m_new = fmaxf(row_m[nb][i], mx - P::kShift);
                        const float alpha = m_new == -INFINITY ? 1.f : ex2(row_m[nb][i] - m_new);
                        row_m[nb][i] = m_new;
                        row_b[nb][i] = m_new == -INFINITY ? 0.f : m_new;
                        row_l[nb][i] *= alpha;
#pragma unroll
                        for (int m = 0; m < MT; m++) acc[m][nb][i] *= alpha, acc[m][nb][2 + i] *= alpha;
                    }
            }
#pragma unroll
            for (int sub = 0; sub < 2; sub++) {
                uint32_t pf[NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; nb++) {
                    float(&x)[4] = s[sub][nb];
#pragma unroll
                    for (int i = 0; i < 4; i++) x[i] = ex2(fmaf(x[i], sc[nb][i & 1], -row_b[nb][i & 1]));
                    row_l[nb][0] += x[0] + x[2];
                    row_l[nb][1] += x[1] + x[3];
                    // P is rounded to halves for the product (down to 2^-25 of the largest); l sums it unrounded
                    pf[nb][0] = transpose8x8(P::pack(x[0], x[1]));
                    pf[nb][1] = transpose8x8(P::pack(x[2], x[3]));
                }
                constexpr int NW = D / 64;   // words of 8 codes per thread and key, all of one block
                uint32_t v[4][NW], sv[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {   // keys 2 cc, 2 cc + 1, 2 cc + 8, 2 cc + 9
                    const uint32_t from = ((i & 1) ? at_v1 : at_v) + (sub * kStep + 8 * (i >> 1)) * C::RB;
                    if constexpr (NW == 2) {
                        const uint2 x = lds64(from);
                        v[i][0] = x.x, v[i][1] = x.y;
                    } else {
                        v[i][0] = lds32(from);
                    }
                    sv[i] = lds_u8(at_vs + (sub * kStep + (i & 1) + 8 * (i >> 1)) * C::SB);
                }
                const uint32_t s01 = e4m3x2_half2(__byte_perm(sv[0], sv[1], 0x0040)), s23 = e4m3x2_half2(__byte_perm(sv[2], sv[3], 0x0040));
#pragma unroll
                for (int u = 0; u < NW; u++) {
                    // the same element's codes of two keys in one byte before the conversion
                    uint32_t e[2][2][4];
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const uint32_t x = v[2 * i][u], y = v[2 * i + 1][u];
                        e2m1x8_half8(low_nibbles_of(x, y << 4), e[0][i]);
                        e2m1x8_half8(low_nibbles_of(x >> 4, y), e[1][i]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const uint32_t a[4] = {hmul2(e[0][0][j], s01), hmul2(e[1][0][j], s01), hmul2(e[0][1][j], s23), hmul2(e[1][1][j], s23)};
#pragma unroll
                        for (int nb = 0; nb < NB; nb++) mma16816<P>(acc[4 * u + j][nb], a, pf[nb][0], pf[nb][1]);
                    }
                }
            }
        };

        int st_in = 0, st_out = 0;
#pragma unroll
        for (int i = 0; i < C::NS - 1; i++) issue(ta + i, st_in++);
        for (int t = ta; t < tb; t++) {
            issue(t + C::NS - 1, st_in);
            st_in = st_in + 1 == C::NS ? 0 : st_in + 1;
            cp_async_wait<C::NS - 1>();
            __syncwarp();
            const int k0 = key_of(t), stage = st_out;
            st_out = st_out + 1 == C::NS ? 0 : st_out + 1;
            if constexpr (KV == kKvE2M1) {
                if (step4_used(k0)) step4(k0, stage);
            } else if (step_used(k0) && !(bad >> stage & 1)) {
                const uint32_t kb = ring + stage * C::STAGE, vb = kb + kStep * C::RB;
                float s[NB][4], s2[NB][4];   // one row block: two chains of products, added at the end
#pragma unroll
                for (int nb = 0; nb < NB; nb++)
#pragma unroll
                    for (int i = 0; i < 4; i++) s[nb][i] = s2[nb][i] = 0.f;
                auto qk = [&](int kb_, const uint32_t *a) {
#pragma unroll
                    for (int nb = 0; nb < NB; nb++) {
                        uint2 q;
                        if constexpr (C::Q_SMEM) q = lds64(q_at + (nb * (D / 16) + kb_) * 256);
                        else q = make_uint2(qf[kb_][0], qf[kb_][1]);
                        mma16816<P>(NB == 1 && (kb_ & 1) ? s2[nb] : s[nb], a, q.x, q.y);
                    }
                };
#pragma unroll
                for (int j = 0; j < C::CH / 4; j++) {
                    const uint4 x = lds128(kb + g * C::RB + (((cc + 4 * j) ^ C::swz_k(g)) * 16));
                    const uint4 y = lds128(kb + (g + 8) * C::RB + (((cc + 4 * j) ^ C::swz_k(g + 8)) * 16));
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
                    if constexpr (CODES) {
#pragma unroll
                        for (int u = 0; u < 4; u++) {
                            uint32_t a[4];
                            e4m3x4_half4(xs[u], a[0], a[2]);
                            e4m3x4_half4(ys[u], a[1], a[3]);
                            qk(4 * j + u, a);
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            const uint32_t a[4] = {xs[2 * u], ys[2 * u], xs[2 * u + 1], ys[2 * u + 1]};
                            qk(2 * j + u, a);
                        }
                    }
                }
                // s[nb]: keys k0 + g (+ 8), rows nb * 8 + 2 cc (+ 1); in units of log2
                const bool all = k0 + kStep - 1 <= p0 && (k0 >= lo_all || k0 + kStep <= S);
                // The maximum is moved (by all of a row's lanes) only when a score passes it by more than kGrow: the
                // usual step has no exchange between lanes.  row_m is kShift below it; P, l and O have its scale.
                bool grown = false;
#pragma unroll
                for (int nb = 0; nb < NB; nb++) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if constexpr (NB == 1) s[nb][i] += s2[nb][i];
                        if (!all && !key_visible(k0 + g + 8 * (i >> 1), row_pos[nb][i & 1], W, S)) s[nb][i] = -INFINITY;
                    }
#pragma unroll
                    for (int i = 0; i < 2; i++) grown |= fmaxf(s[nb][i], s[nb][i + 2]) * sc[nb][i] > row_m[nb][i] + (P::kShift + P::kGrow);
                }
                if (__any_sync(~0u, grown)) {
#pragma unroll
                    for (int nb = 0; nb < NB; nb++)
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            float mx = fmaxf(s[nb][i], s[nb][i + 2]);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
                            const float m_new = fmaxf(row_m[nb][i], mx * sc[nb][i] - P::kShift);
                            const float alpha = m_new == -INFINITY ? 1.f : ex2(row_m[nb][i] - m_new);
                            row_m[nb][i] = m_new;
                            row_l[nb][i] *= alpha;
#pragma unroll
                            for (int m = 0; m < MT; m++) acc[m][nb][i] *= alpha, acc[m][nb][2 + i] *= alpha;
                        }
                }
                uint32_t pf[NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; nb++) {
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float base = row_m[nb][i] == -INFINITY ? 0.f : row_m[nb][i];   // a row that has seen no key yet
                        s[nb][i] = ex2(fmaf(s[nb][i], sc[nb][i], -base));
                        s[nb][i + 2] = ex2(fmaf(s[nb][i + 2], sc[nb][i], -base));
                        row_l[nb][i] += s[nb][i] + s[nb][i + 2];
                    }
                    // P is rounded to the product's 16-bit type (relative error 2^-8 or 2^-11, as the
                    // output's own rounding; halves: down to 2^-25 of the largest); l sums it unrounded
                    pf[nb][0] = transpose8x8(P::pack(s[nb][0], s[nb][1]));
                    pf[nb][1] = transpose8x8(P::pack(s[nb][2], s[nb][3]));
                }
                const int kk[4] = {2 * cc, 2 * cc + 1, 2 * cc + 8, 2 * cc + 9};
                auto pv = [&](int m, const uint32_t v0, const uint32_t v1, const uint32_t v2, const uint32_t v3) {
                    const uint32_t a[4] = {__byte_perm(v0, v1, 0x5410), __byte_perm(v0, v1, 0x7632),
                                           __byte_perm(v2, v3, 0x5410), __byte_perm(v2, v3, 0x7632)};
#pragma unroll
                    for (int nb = 0; nb < NB; nb++) mma16816<P>(acc[m][nb], a, pf[nb][0], pf[nb][1]);
                };
                if constexpr (!CODES) {
#pragma unroll
                    for (int hh = 0; hh < D / 64; hh++) {
                        uint32_t v[4][4];
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const uint4 x = lds128(vb + kk[i] * C::RB + (((8 * hh + g) ^ C::swz_v(kk[i])) * 16));
                            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
                        }
#pragma unroll
                        for (int i = 0; i < 4; i++) pv(4 * hh + i, v[0][i], v[1][i], v[2][i], v[3][i]);
                    }
                } else {
                    constexpr int NW = D / 32;   // words of 4 codes per thread and key
                    uint32_t v[4][NW];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if constexpr (NW == 4) {
                            const uint4 x = lds128(vb + kk[i] * C::RB + ((g ^ C::swz_v(kk[i])) * 16));
                            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
                        } else {
                            const uint2 x = lds64(vb + kk[i] * C::RB + (((g >> 1) ^ C::swz_v(kk[i])) * 16) + 8 * (g & 1));
                            v[i][0] = x.x, v[i][1] = x.y;
                        }
                    }
#pragma unroll
                    for (int u = 0; u < NW; u++) {
                        // codes of two keys side by side before the conversion: (a0 b0 a1 b1), (a2 b2 a3 b3)
                        uint32_t e[2][4];
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            e4m3x4_half4(__byte_perm(v[2 * i][u], v[2 * i + 1][u], 0x5140), e[0][2 * i], e[0][2 * i + 1]);
                            e4m3x4_half4(__byte_perm(v[2 * i][u], v[2 * i + 1][u], 0x7362), e[1][2 * i], e[1][2 * i + 1]);
                        }
#pragma unroll
                        for (int hf = 0; hf < 2; hf++)
#pragma unroll
                            for (int nb = 0; nb < NB; nb++) mma16816<P>(acc[2 * u + hf][nb], e[hf], pf[nb][0], pf[nb][1]);
                    }
                }
            }
            __syncwarp();   // the stage is read: the next issue may overwrite it
        }
        cp_async_wait<0>();

        // ---- the four warps' (m, l, O) into one
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) row_l[nb][i] += __shfl_xor_sync(~0u, row_l[nb][i], o);
        __syncthreads();   // every warp is done with its ring
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int r = nb * 8 + 2 * cc + i;
                if (g == 0) {
                    mg_m[w * ROWS + r] = row_m[nb][i];
                    mg_l[w * ROWS + r] = row_l[nb][i];
                }
                if (r < n_rows) {
#pragma unroll
                    for (int m = 0; m < MT; m++)
                        *reinterpret_cast<float2 *>(&mg[(w * ROWS + r) * D + C::dim(m, g)]) = make_float2(acc[m][nb][i], acc[m][nb][2 + i]);
                }
            }
        __syncthreads();

        const int f = (int)div_pos(u0, chunk), l = (int)div_pos(u0 + kt - 1, chunk);   // CTAs that hold the unit's pieces
        const float v_scale = CODES ? c.v_scale[p.layer * c.Hkv + h] : 1.f;
        auto store = [&](int r, int d, float4 o, float l_sum, float m) {   // 4 outputs of a row
            const int t = (mb * ROWS + r) / p.G, hq = h * p.G + (mb * ROWS + r) % p.G;
            const size_t row = ((size_t)b * p.T + t) * p.Hq + hq;
            const float inv = l_sum == 0.f ? 0.f : v_scale / l_sum;
            // a row that saw no key holds only zeros: 0 * 0
            *reinterpret_cast<uint2 *>(p.out + row * D + d) = make_uint2(Q::pack(o.x * inv, o.y * inv), Q::pack(o.z * inv, o.w * inv));
            if (p.lse && d == 0) p.lse[row] = l_sum == 0.f ? -INFINITY : (m + log2f(l_sum)) * kLn2;
        };
        float *slot = part.slot((int)blockIdx.x * 2 + (f == (int)blockIdx.x), D);
        for (int x = tid; x < n_rows * (D / 4); x += kThreads) {
            const int r = x / (D / 4), d = x % (D / 4) * 4;
            float m = -INFINITY, ls = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; i++) m = fmaxf(m, mg_m[i * ROWS + r]);
            const float base = m == -INFINITY ? 0.f : m;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kWarps; i++) {
                const float a = ex2(mg_m[i * ROWS + r] - base);
                const float4 y = *reinterpret_cast<const float4 *>(&mg[(i * ROWS + r) * D + d]);
                ls += a * mg_l[i * ROWS + r];
                o.x += a * y.x, o.y += a * y.y, o.z += a * y.z, o.w += a * y.w;
            }
            if (f == l) store(r, d, o, ls, m);
            else {
                __stcg(reinterpret_cast<float4 *>(slot + 2 * kUnitRows + r * D + d), o);
                if (d == 0) {
                    __stcg(slot + r, m);
                    __stcg(slot + kUnitRows + r, ls);
                }
            }
        }
        if (f != l) {
            // pieces [i0, i1) (i-th piece: the unit's slot of CTA f + i, one in `step` of them) in order
            auto join = [&](int i0, int i1, int step, bool last) {
                float *to = part.slot(2 * (f + i0) + (i0 == 0), D);
                for (int x = tid; x < n_rows * (D / 4); x += kThreads) {
                    const int r = x / (D / 4), d = x % (D / 4) * 4;
                    float m = -INFINITY, ls = 0.f;
#pragma unroll 8
                    for (int i = i0; i < i1; i += step) m = fmaxf(m, __ldcg(part.slot(2 * (f + i) + (i == 0), D) + r));
                    const float base = m == -INFINITY ? 0.f : m;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int i = i0; i < i1; i += step) {
                        const float *q = part.slot(2 * (f + i) + (i == 0), D);
                        const float a = ex2(__ldcg(q + r) - base);
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(q + 2 * kUnitRows + r * D + d));
                        ls += a * __ldcg(q + kUnitRows + r);
                        o.x += a * y.x, o.y += a * y.y, o.z += a * y.z, o.w += a * y.w;
                    }
                    if (last) store(r, d, o, ls, m);
                    else {
                        __stcg(reinterpret_cast<float4 *>(to + 2 * kUnitRows + r * D + d), o);
                        // the row's (m, l) are still read by its other threads: kept apart until all are done
                        if (d == 0) mg_m[r] = m, mg_l[r] = ls;
                    }
                }
                if (!last) {
                    __syncthreads();
                    if (tid < n_rows) {
                        __stcg(to + tid, mg_m[tid]);
                        __stcg(to + kUnitRows + tid, mg_l[tid]);
                    }
                }
            };
            // true in the CTA that is the `n`-th to come to this counter, which is then ready for the next call
            auto last_of = [&](int *counter, int n) {
                __threadfence();
                __syncthreads();
                if (tid == 0) {
                    const int done = atomicAdd(counter, 1);
                    sh_last = done == n - 1;
                    if (sh_last) *counter = 0;
                    __threadfence();
                }
                __syncthreads();
                return sh_last != 0;
            };
            // up to 16 pieces are joined at once, more in groups of 8 first
            const int n = l - f + 1;
            if (n <= 16) {
                if (last_of(&part.count[f], n)) join(0, n, 1, true);
            } else {
                const int i0 = ((int)blockIdx.x - f) & ~7, i1 = min(n, i0 + 8);
                if (last_of(&part.group[2 * (f + i0) + (i0 == 0)], i1 - i0)) {
                    join(i0, i1, 1, false);
                    if (last_of(&part.count[f], (n + 7) / 8)) join(0, n, 8, true);
                }
            }
        }
        __syncthreads();   // the merge buffer is read: the next run's copies may land in it
        at = u0 + tb;
    }
}

template <int D, typename Q, int KV, int NB>
cudaError_t launch_as(const AttnParams &p, cudaStream_t stream)
{
    static KernelSetup setup;
    constexpr int smem = Cfg<D, KV, NB>::SMEM;
    static_assert(Cfg<D, KV, NB>::NS >= 2 && Cfg<D, KV, NB>::NS <= 16, "a ring of two stages at least");
    int resident = 0;
    const cudaError_t e = setup.get(kda_attn_decode_kernel<D, Q, KV, NB>, kThreads, smem, 0, &resident);
    if (e != cudaSuccess) return e;
    if (resident < 1) return cudaErrorLaunchOutOfResources;
    return launch_pdl(kda_attn_decode_kernel<D, Q, KV, NB>, dim3((unsigned)min(resident, kMaxCtas)), dim3(kThreads), smem, stream, p);
}

// Row blocks of 8, 16, 24 or 32: the smallest that holds the rows of a sequence and key head, at most 32
// (more rows read the keys again from L2).  A step's instructions grow with the block: 20 rows, 64 sequences in
// a 1024 window: 41 us with 32, 36 us with 24 (and without the second
// chain of products and the separate scaling that both had).
template <int D, typename Q, int KV>
cudaError_t launch_rows(const AttnParams &p, cudaStream_t stream)
{
    const int rows = p.T * p.G;
    if (rows <= 8) return launch_as<D, Q, KV, 1>(p, stream);
    if (rows <= 16) return launch_as<D, Q, KV, 2>(p, stream);
    if (rows <= 24) return launch_as<D, Q, KV, 3>(p, stream);
    return launch_as<D, Q, KV, 4>(p, stream);
}

template <int D, int KV>
cudaError_t launch_types(const AttnParams &p, cudaStream_t stream)
{
    return p.f16 ? launch_rows<D, Half, KV>(p, stream) : launch_rows<D, Bf16, KV>(p, stream);
}

}  // namespace
}  // namespace kda
