// kda_attn_prefill.cu -- attention of packed new tokens over a paged key-value cache
// (kda_attn_prefill), on the 5th-generation tensor cores.
//
// Mathematics.  The rows of one sequence and key head are its (token, query head) pairs in that
// order; a CTA takes 256 of them as two halves of 128 and walks the key tiles (128 keys) that its
// tokens see.  Per half and tile: S = Q K^T into tensor memory, one thread per row takes the row's
// maximum, P = exp2(S - m) back into tensor memory in 16 bits, O += P V with P as the tensor-memory
// operand.  The running maximum m is only moved (and O rescaled) when it grows by more than 2^8: P
// then stays below 2^8, which both 16-bit types hold with their full relative precision, and l and
// O are FP32 sums of the same scale.
//
// Bound.  4 D flops for each visible (row, key) pair against D bytes moved once per 256 rows: the
// tensor cores, or the 128 x 128 exponentials of each tile next to them.  Two halves, so that one
// half's softmax runs while the tensor cores work on the other's products.
//
// Roles: warps 0-3 and 4-7 are the softmax of the two halves (one thread per row), warps 8-11 copy
// keys and values into a ring of shared-memory tiles, one lane of warp 12 issues every MMA (warps 13-15
// only give their registers away).  Hand-over
// by mbarriers; a half's S tile also orders its previous P V (a commit covers every MMA issued before
// it).  With few row tiles the key tiles are split over several CTAs whose partial (m, l, O) the last
// one to finish joins in a fixed order.
//
// Tiles are stored with the 128-byte swizzle, 64 head dims wide: row r, 16-byte chunk g of half c at
// c 16 KiB + r 128 + (g ^ r % 8) 16.  Read along head dims that is the K-major operand of Q K^T, read
// along keys the MN-major operand of P V, so keys and values are stored alike.  A tile whose keys are all
// seen by some token of the CTA comes by TMA, one box for each page and half; at the ends of the range
// the loader threads copy it themselves and write zeros for the keys that no token sees, so that
// whatever the page holds there (NaN included) cannot reach the products.  The same threads convert E4M3
// codes on their way.
#include <cuda.h>

#include "kda_attn_common.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kHalf = 128, kRowsCta = 256, kKeys = 128;
constexpr int kSoftmax = 256, kLoaders = 128, kThreads = kSoftmax + kLoaders + 128;
// Registers of a thread: all start with 128 (512 threads, the whole file), then the softmax holds a row
// of S at once, the loaders two fetches of E4M3 codes; 256 x 184 + 128 x 104 + 128 x 40 = 65536.
constexpr int kRegs = 128, kRegsSoftmax = 184, kRegsLoad = 104, kRegsMma = 40;
constexpr int kSlots = 4, kHalfBytes = kKeys * 128;   // a tile's 64 head dims: 128 rows of 128 bytes
constexpr int kMaxSplitCtas = 256;             // CTAs of a launch whose keys are split
constexpr uint64_t kLimitNs = 2000000000ull;   // bound of every wait
constexpr float kGrow = 8.f;                   // log2 growth of the maximum that O is rescaled for

template <int D>
struct Smem {
    uint8_t q[2][kHalf * D * 2];
    uint8_t kv[kSlots][kKeys * D * 2];
    uint64_t q_full, full[kSlots], empty[kSlots], s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem;
    int unit_b, unit_tile, c0, n, last;
    volatile int stop;
};

struct Args {
    AttnParams p;
    CUtensorMap k, v;   // [layers pages][Hkv page_size][D], boxes of one page's tokens x 64 head dims
};

// Byte offset of 16-byte chunk g (of the row's D / 8) of row r in a tile.
__device__ __forceinline__ int chunk_at(int r, int g) { return (g >> 3) * kHalfBytes + r * 128 + (((g & 7) ^ (r & 7)) << 4); }

// Shared-memory matrix descriptor with the 128-byte swizzle: groups of 8 rows are 1024 bytes apart;
// `lbo`: step between 64-element groups along a contiguous (MN-major) dimension.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo)
{
    return (uint64_t)((saddr >> 4) & 0x3fffu) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}

// Tensor memory columns: S of both halves, O of both halves; P takes the place of S (the next S
// of a half is issued after the P V that reads P; both products then have the same shape), or
// columns of its own where head_dim 64 leaves some.
template <int D>
struct Cols {
    static constexpr int s(int h) { return h * 128; }
    static constexpr int o(int h) { return 256 + h * D; }
    static constexpr int p(int h) { return D == 128 ? s(h) : 384 + h * 64; }
};

__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

static_assert(kSoftmax * kRegsSoftmax + kLoaders * kRegsLoad + 128 * kRegsMma <= kThreads * kRegs, "setmaxnreg would wait forever");

// 32 tensor-memory columns of this warp's lanes.  Load and wait are one statement, so that nothing
// that uses the registers can be placed between them.
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a) : "memory");
}
// ... without the wait.
__device__ __forceinline__ void tmem_ld32_async(uint32_t a, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a) : "memory");
}
// Waits for this thread's tensor-memory loads; the 32 registers pass through, so that what uses them comes after.
__device__ __forceinline__ void tmem_wait_ld(uint32_t *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
        :: "memory");
}
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1)
{
    asm("{\n\t.reg .b64 a, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 d, {%0, %1};\n\tadd.rn.f32x2 d, d, a;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1));
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
          "r"(a) : "memory");
}
template <typename Q>
__host__ __device__ constexpr uint32_t idesc(int N)
{
    return Q::is_half ? (tc::idesc_bf16(128, N) & ~((1u << 7) | (1u << 10))) : tc::idesc_bf16(128, N);
}

// D (+)= A B with A [128 x 16] in tensor memory (16-bit pairs along K, 8 columns)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t id, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b_desc), "r"(id), "r"((uint32_t)accumulate)
        : "memory");
}

// What a CTA works on.
struct Unit {
    int row;               // cache row
    int h;                 // key head
    int b, c0, n, len;     // sequence, first packed token, new tokens, row length
    int r0, rows;          // rows [r0, r0 + rows) of the sequence's n * G
    int halves;
    int ta, tb;            // key tiles of the range that this CTA takes
};

template <int D>
__device__ __forceinline__ bool wait(Smem<D> &sm, uint64_t *bar, uint32_t parity, int *err)
{
    if (mbar_wait_bounded(bar, parity, kLimitNs)) return true;
    sm.stop = 1;
    atomicOr(err, KDA_DEVERR_TIMEOUT);
    return false;
}
// ... by all lanes of a warp, which agree on the outcome
template <int D>
__device__ __forceinline__ bool wait_warp(Smem<D> &sm, uint64_t *bar, uint32_t parity, int *err)
{
    return __all_sync(~0u, wait(sm, bar, parity, err));
}

// ---- warp 12: products, in the order that lets one half's softmax run beside the other's products
template <int D, typename Q>
__device__ void issue_products(Smem<D> &sm, const Unit &u, uint32_t tmem, int *err)
{
    const int n = u.tb - u.ta;
    auto slot_wait = [&](int item) { return wait(sm, &sm.full[item % kSlots], (item / kSlots) & 1, err); };
    auto qk = [&](int h, int item) {
        const uint64_t ad = desc_sw128(smem_u32(sm.q[h]), 16u), bd = desc_sw128(smem_u32(sm.kv[item % kSlots]), 16u);
#pragma unroll
        for (int k = 0; k < D / 16; k++) {   // 16 head dims: 32 bytes further in the half's rows
            const uint32_t step = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
            tc::mma(tmem + Cols<D>::s(h), ad + step, bd + step, idesc<Q>(kKeys), k > 0);
        }
        tc::commit(&sm.s_full[h]);
    };
    auto pv = [&](int h, int item, bool accumulate) {
        const uint64_t bd = desc_sw128(smem_u32(sm.kv[item % kSlots]), kHalfBytes);
#pragma unroll
        for (int k = 0; k < kKeys / 16; k++)   // 16 keys: two groups of 8 rows
            mma_ts(tmem + Cols<D>::o(h), tmem + Cols<D>::p(h) + 8 * k, bd + k * (2048u >> 4), idesc<Q>(D) | (1u << 16), accumulate || k > 0);
    };
    if (!wait(sm, &sm.q_full, 0, err)) return;
    if (!slot_wait(0)) return;
    tc::fence_after_sync();
    for (int h = 0; h < u.halves; h++) qk(h, 0);
    tc::commit(&sm.empty[0]);
    for (int i = 0; i < n; i++) {
        if (!slot_wait(2 * i + 1)) return;
        for (int h = 0; h < u.halves; h++) {
            if (!wait(sm, &sm.p_full[h], i & 1, err)) return;
            tc::fence_after_sync();
            pv(h, 2 * i + 1, i > 0);
            if (i + 1 == n) tc::commit(&sm.o_full[h]);
            if (h + 1 == u.halves) tc::commit(&sm.empty[(2 * i + 1) % kSlots]);
            if (i + 1 < n) {
                if (h == 0) {
                    if (!slot_wait(2 * i + 2)) return;
                    tc::fence_after_sync();
                }
                qk(h, 2 * i + 2);
                if (h + 1 == u.halves) tc::commit(&sm.empty[(2 * i + 2) % kSlots]);
            }
        }
    }
}

// ---- warps 8-11: keys and values of tile i as ring items 2 i and 2 i + 1
template <int D, typename Q, bool FP8>
__device__ void load_tiles(Smem<D> &sm, const Args &args, const Unit &u, const KeyRange<kKeys> &kr, int S)
{
    const AttnParams &p = args.p;
    const PagedCache &c = p.c;
    const int tid = threadIdx.x - kSoftmax, w = tid >> 5, lane = tid & 31, r8 = lane & 7, q4 = lane >> 3;
    const int n = u.tb - u.ta;
    constexpr int ES = FP8 ? 1 : 2, RB = D * ES;
    constexpr int CPR = RB / 16;              // 16-byte chunks of a key
    constexpr int PASS = CPR / 4;             // passes of four chunks over a group of 8 keys
    constexpr int GR = kKeys / 8 / 4;         // groups of 8 keys of a warp: w, w + 4, ...
    const size_t head_bytes = (size_t)c.ps * RB;
    // page of key group `lane` (16 groups of a tile), -1: none of its keys is seen
    auto pages_of = [&](int i) {
        const int k0 = kr.tile(u.ta + i) * kKeys + lane * 8;
        if (i >= n || lane >= kKeys / 8 || k0 >= kr.end || !(k0 + 8 > kr.lo || k0 < S)) return -1;
        return __ldg(c.table + (size_t)u.row * c.width + (k0 >> c.ps_log2));
    };
    int pages = pages_of(0), pages_next = pages_of(1);
    // source of this lane's key of group gi of tile i; null where nothing is read
    auto source = [&](const uint8_t *base, int i, int gi, int pg) -> const uint8_t * {
        const int k0 = kr.tile(u.ta + i) * kKeys + gi * 8, j = k0 + r8;
        if (!(j < kr.end && (j >= kr.lo || j < S))) return nullptr;
        if ((unsigned)pg >= (unsigned)c.pages) {
            atomicOr(c.err, KDA_DEVERR_PAGE);
            return nullptr;
        }
        return base + (((size_t)p.layer * c.pages + pg) * c.Hkv + u.h) * head_bytes + (size_t)(j & (c.ps - 1)) * RB;
    };
    if constexpr (!FP8) {
        for (int it = 0; it < 2 * n; it++) {
            const int i = it >> 1, slot = it % kSlots, k0 = kr.tile(u.ta + i) * kKeys;
            const uint8_t *base = it & 1 ? c.v : c.k;
            // every key is seen by some token and has a page (the four warps hold the same page ids)
            const bool whole = k0 + kKeys <= kr.end && (k0 >= kr.lo || k0 + kKeys <= S) &&
                               __all_sync(~0u, lane >= kKeys / 8 || (unsigned)pages < (unsigned)c.pages);
            if (it >= kSlots && !wait_warp(sm, &sm.empty[slot], (it / kSlots - 1) & 1, c.err)) break;
            if (whole) {
                if (w == 0) {
                    if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], kKeys * RB);
                    __syncwarp();
                    // lane: page and half of the tile
                    const int boxes = kKeys >> c.ps_log2, x = lane / boxes, y = lane % boxes;
                    const int page = __shfl_sync(~0u, pages, y << (c.ps_log2 - 3));
                    if (x < D / 64)
                        tma_load_3d(smem_u32(sm.kv[slot]) + x * kHalfBytes + (y << c.ps_log2) * 128, it & 1 ? &args.v : &args.k,
                                    x * 64, u.h << c.ps_log2, p.layer * c.pages + page, &sm.full[slot]);
                    if (lane > 0) mbar_arrive(&sm.full[slot]);
                } else {
                    mbar_arrive(&sm.full[slot]);
                }
            } else {
#pragma unroll
                for (int a = 0; a < GR; a++) {
                    const int gi = w + 4 * a;
                    const uint8_t *src = source(base, i, gi, __shfl_sync(~0u, pages, gi));
#pragma unroll
                    for (int x = 0; x < PASS; x++)
                        cp_async16(sm.kv[slot] + chunk_at(gi * 8 + r8, x * 4 + q4), src ? src + (x * 4 + q4) * 16 : c.k, src ? 16 : 0);
                }
                cp_async_wait_all();
                tc::fence_smem_to_async();
                mbar_arrive(&sm.full[slot]);
            }
            if (it & 1) {
                pages = pages_next;
                pages_next = pages_of(i + 2);
            }
        }
    } else {
        // codes pass through registers: the next item's loads are in flight while this one's are
        // converted (exactly) to the query's type and stored
        uint4 cur[GR * PASS > 0 ? GR * PASS : 1], nxt[GR * PASS > 0 ? GR * PASS : 1];
        auto fetch = [&](int it, uint4 *v, int pg_lane) {
            const uint8_t *base = it & 1 ? c.v : c.k;
#pragma unroll
            for (int a = 0; a < GR; a++) {
                const int gi = w + 4 * a;
                const uint8_t *src = source(base, it >> 1, gi, __shfl_sync(~0u, pg_lane, gi));
#pragma unroll
                for (int x = 0; x < PASS; x++)
                    v[a * PASS + x] = src ? __ldg(reinterpret_cast<const uint4 *>(src + (x * 4 + q4) * 16)) : make_uint4(0, 0, 0, 0);
            }
        };
        fetch(0, cur, pages);
        for (int it = 0; it < 2 * n; it++) {
            const int slot = it % kSlots;
            if (it + 1 < 2 * n) {
                if (it & 1) {
                    pages = pages_next;
                    pages_next = pages_of((it >> 1) + 2);
                }
                fetch(it + 1, nxt, pages);
            }
            if (it >= kSlots && !wait_warp(sm, &sm.empty[slot], (it / kSlots - 1) & 1, c.err)) break;
#pragma unroll
            for (int a = 0; a < GR; a++)
#pragma unroll
                for (int x = 0; x < PASS; x++) {
                    const uint4 v = cur[a * PASS + x];
                    const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int s = 0; s < 2; s++)
                        *reinterpret_cast<uint4 *>(sm.kv[slot] + chunk_at((w + 4 * a) * 8 + r8, (x * 4 + q4) * 2 + s)) =
                            make_uint4(e4m3x2_as<Q>(ws[2 * s], 0), e4m3x2_as<Q>(ws[2 * s], 1), e4m3x2_as<Q>(ws[2 * s + 1], 0), e4m3x2_as<Q>(ws[2 * s + 1], 1));
                }
            tc::fence_smem_to_async();
            mbar_arrive(&sm.full[slot]);
#pragma unroll
            for (int a = 0; a < GR * PASS; a++) cur[a] = nxt[a];
        }
    }
}

struct SplitWs {   // partial results of split units: (m, l) and O by column, so that threads (rows) are contiguous
    float *data;
    static constexpr size_t slot_floats(int D) { return (size_t)kRowsCta * (D + 2); }
    __device__ float *slot(int s, int D) const { return data + (size_t)s * slot_floats(D); }
};

template <typename Q>
__device__ __forceinline__ void store_row(const AttnParams &p, const Unit &u, int r, int d, const float *o, float f)
{
    const int tok = u.c0 + r / p.G, hq = u.h * p.G + r % p.G;
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + ((size_t)tok * p.Hq + hq) * p.c.D + d);
#pragma unroll
    for (int i = 0; i < 4; i++)
        dst[i] = make_uint4(Q::pack(o[8 * i] * f, o[8 * i + 1] * f), Q::pack(o[8 * i + 2] * f, o[8 * i + 3] * f),
                            Q::pack(o[8 * i + 4] * f, o[8 * i + 5] * f), Q::pack(o[8 * i + 6] * f, o[8 * i + 7] * f));
}

// ---- warps 0-7: one thread per row
template <int D, typename Q, bool FP8>
__device__ void softmax_rows(Smem<D> &sm, const AttnParams &p, const Unit &u, const KeyRange<kKeys> &kr, uint32_t tmem, int W, int S,
                             float *partial)
{
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, h = tid >> 7, rl = tid & 127, w = tid >> 5;
    const int n = u.tb - u.ta;
    const int r = u.r0 + h * kHalf + rl;                         // row of the sequence
    const bool live = h * kHalf + rl < u.rows;
    // this row's queries into shared memory
    if (h < u.halves) {
        const uint16_t *src = p.q + (long long)(u.c0 + r / p.G) * p.ql.token + (long long)(u.h * p.G + r % p.G) * p.ql.head;
#pragma unroll
        for (int g = 0; g < D / 8; g++)
            *reinterpret_cast<uint4 *>(sm.q[h] + chunk_at(rl, g)) = live ? __ldg(reinterpret_cast<const uint4 *>(src) + g) : make_uint4(0, 0, 0, 0);
        tc::fence_smem_to_async();
    }
    mbar_arrive(&sm.q_full);
    if (h >= u.halves) return;
    // (a scale of 0 as the least that keeps hidden scores at -inf)
    const float sc = fmaxf(p.scale_log2 * (FP8 ? c.k_scale[p.layer * c.Hkv + u.h] : 1.f), 1e-37f);
    const int first = u.len - u.n;
    const int pos = first + min(r, u.n * p.G - 1) / p.G;          // this row's position
    const int lo = (int)max(-0x7fffffffll, (long long)pos - W + 1);
    // positions of the half's first and last row: whether a tile is seen by all of it
    const int p_lo = first + (u.r0 + h * kHalf) / p.G, p_hi = first + min(u.r0 + h * kHalf + kHalf - 1, u.n * p.G - 1) / p.G;
    const long long lo_all = (long long)p_hi - W + 1;
    const uint32_t lane_base = tmem + ((uint32_t)(w & 3) * 32u << 16);
    const uint32_t ts = lane_base + Cols<D>::s(h), tp = lane_base + Cols<D>::p(h), to = lane_base + Cols<D>::o(h);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int i = 0; i < n; i++) {
        const int k0 = kr.tile(u.ta + i) * kKeys;
        const bool all = k0 + kKeys - 1 <= p_lo && (k0 >= lo_all || k0 + kKeys <= S);
        if (!(ok = wait_warp(sm, &sm.s_full[h], i & 1, c.err))) break;
        tc::fence_after_sync();
        uint32_t v[kKeys];
#pragma unroll
        for (int q = 0; q < 4; q++) tmem_ld32_async(ts + 32 * q, v + 32 * q);
#pragma unroll
        for (int q = 0; q < 4; q++) tmem_wait_ld(v + 32 * q);
        if (!all) {
            const int hi_j = pos - k0, lo_j = max(lo, k0) - k0, s_j = S - k0;
#pragma unroll
            for (int j = 0; j < kKeys; j++)
                if (!(j <= hi_j && (j >= lo_j || j < s_j))) v[j] = 0xff800000u;   // -inf
        }
        float mx0 = __uint_as_float(v[0]), mx1 = __uint_as_float(v[1]);
#pragma unroll
        for (int j = 2; j < kKeys - 2; j += 4) {
            mx0 = fmaxf(mx0, fmaxf(__uint_as_float(v[j]), __uint_as_float(v[j + 1])));
            mx1 = fmaxf(mx1, fmaxf(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])));
        }
        const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(__uint_as_float(v[kKeys - 2]), __uint_as_float(v[kKeys - 1])));
        const float m_new = fmaxf(m, mx * sc);
        if (i == 0) m = m_new;
        else if (__any_sync(~0u, m_new > m + kGrow)) {
            // the products that wrote O are done: this tile's S was issued after them
            const float a = m_new == -INFINITY ? 1.f : ex2(m - m_new);
            l *= a;
            m = m_new;
#pragma unroll 1
            for (int q = 0; q < D / 32; q++) {
                uint32_t o[32];
                tmem_ld32(to + 32 * q, o);
#pragma unroll
                for (int j = 0; j < 32; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
                tmem_st32(to + 32 * q, o);
            }
        }
        const float base = m == -INFINITY ? 0.f : m;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int q = 0; q < 2; q++) {
#pragma unroll
            for (int j = 64 * q; j < 64 * q + 64; j += 2) {
                float e0, e1;
                tc::fma2(e0, e1, __uint_as_float(v[j]), __uint_as_float(v[j + 1]), sc, sc, -base, -base);
                e0 = ex2(e0);
                e1 = ex2(e1);
                add2(s0, s1, e0, e1);
                v[j / 2] = Q::pack(e0, e1);   // rounded to 16 bits for the product; l sums it unrounded
            }
            tmem_st32(tp + 32 * q, v + 32 * q);
        }
        l += s0 + s1;
        tmem_wait_st();
        tc::fence_before_sync();
        mbar_arrive(&sm.p_full[h]);
    }
    if (ok) ok = wait_warp(sm, &sm.o_full[h], 0, c.err);
    tc::fence_after_sync();
    if (!ok) return;
    const float f = l == 0.f ? 0.f : (FP8 ? c.v_scale[p.layer * c.Hkv + u.h] : 1.f) / l;
#pragma unroll 1
    for (int q = 0; q < D / 32; q++) {
        uint32_t v[32];
        tmem_ld32(to + 32 * q, v);
        if (partial) {
#pragma unroll
            for (int j = 0; j < 32; j++) __stcg(partial + (2 + 32 * q + j) * kRowsCta + tid, __uint_as_float(v[j]));
        } else if (live) {
            store_row<Q>(p, u, r, 32 * q, reinterpret_cast<const float *>(v), f);
        }
    }
    if (partial) {
        __stcg(partial + tid, m);
        __stcg(partial + kRowsCta + tid, l);
    } else if (live && p.lse) {
        p.lse[(size_t)(u.c0 + r / p.G) * p.Hq + u.h * p.G + r % p.G] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

template <int D, typename Q, bool FP8>
__global__ void __launch_bounds__(kThreads, 1) kda_attn_prefill_kernel(const __grid_constant__ Args args)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // the swizzle repeats every 1024 bytes of the shared address
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const AttnParams &p = args.p;
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int W = p.window > 0 ? p.window : 0x7fffffff, S = p.window > 0 ? p.sinks : 0;
    const int splits = gridDim.y;
    if (tid == 0) {
        mbar_init(&sm.q_full, kSoftmax);
        mbar_init(&sm.drain, 1);
        for (int i = 0; i < kSlots; i++) {
            mbar_init(&sm.full[i], kLoaders);
            mbar_init(&sm.empty[i], 1);
        }
        for (int h = 0; h < 2; h++) {
            mbar_init(&sm.s_full[h], 1);
            mbar_init(&sm.p_full[h], kHalf);
            mbar_init(&sm.o_full[h], 1);
        }
        sm.stop = 0;
        sm.unit_b = -1;
        fence_mbar_init();
    }
    __syncthreads();
    grid_dependency_wait();

    // ---- which sequence and row tile: the CTAs count the tiles from the last one back, so that the
    // longest ones of a causal prompt start first
    if (warp == 0) {
        const int x = blockIdx.x / c.Hkv;
        const bool report = blockIdx.x == 0 && blockIdx.y == 0;
        int before = 0, all = 0;
        for (int pass = 0; pass < 2; pass++) {   // first the number of tiles, then the tile (in one go up to 32 sequences)
            int want = all - 1 - x;
            if (pass == 1 && want < 0) break;
            before = 0;
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int b = b0 + lane;
                int tiles = 0, c0 = 0, n = 0;
                if (b < p.B) {
                    c0 = p.cu[b];
                    const int c1 = p.cu[b + 1], row = p.rows[b];
                    if (c0 < 0 || c1 < c0 || c1 > p.total || c1 - c0 > p.T || (b > 0 && p.cu[b - 1] > c0)) {
                        if (report && pass == 0) atomicOr(c.err, KDA_DEVERR_SEQLEN);
                    } else if (c1 > c0 && seq_info(c, row, c1 - c0, 0x7fffffff, report && pass == 0).ok) n = c1 - c0;
                    tiles = (n * p.G + kRowsCta - 1) / kRowsCta;
                }
                int inc = tiles;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(~0u, inc, o);
                    if (lane >= o) inc += y;
                }
                const int sum = __shfl_sync(~0u, inc, 31);
                if (p.B <= 32) want = sum - 1 - x;
                if ((pass == 1 || p.B <= 32) && want >= before + inc - tiles && want < before + inc) {
                    sm.unit_b = b;
                    sm.unit_tile = want - (before + inc - tiles);
                    sm.c0 = c0;
                    sm.n = n;
                }
                before += sum;
            }
            all = before;
            if (p.B <= 32) break;
        }
    }
    __syncthreads();
    Unit u;
    u.b = sm.unit_b;
    if (u.b < 0) return;
    u.h = blockIdx.x % c.Hkv;
    u.c0 = sm.c0;
    u.n = sm.n;
    u.row = p.rows[u.b];
    u.len = c.lens[u.row];
    u.r0 = sm.unit_tile * kRowsCta;
    u.rows = min(kRowsCta, u.n * p.G - u.r0);
    u.halves = u.rows > kHalf ? 2 : 1;
    const int first = u.len - u.n;
    const KeyRange<kKeys> kr(first + u.r0 / p.G, first + (u.r0 + u.rows - 1) / p.G, u.len, W, S);
    // this CTA's share of the key tiles, two at least (a unit without keys has one CTA and no tile)
    const int share = max(2, (kr.count + splits - 1) / splits), pieces = max(1, (kr.count + share - 1) / share);
    if ((int)blockIdx.y >= pieces) return;
    u.ta = blockIdx.y * share;
    u.tb = min(kr.count, u.ta + share);
    int *count = reinterpret_cast<int *>(p.ws) + blockIdx.x;
    SplitWs ws;
    ws.data = reinterpret_cast<float *>(p.ws + kMaxSplitCtas * sizeof(int));
    float *partial = pieces > 1 ? ws.slot(blockIdx.x * splits + blockIdx.y, D) : nullptr;

    if (kr.count == 0) {   // no token of the tile sees a key
        for (int x = tid; x < u.rows * (D / 32); x += kThreads) {
            const float z[32] = {};
            const int r = u.r0 + x / (D / 32);
            store_row<Q>(p, u, r, x % (D / 32) * 32, z, 0.f);
            if (p.lse && x % (D / 32) == 0) p.lse[(size_t)(u.c0 + r / p.G) * p.Hq + u.h * p.G + r % p.G] = -INFINITY;
        }
        return;
    }

    if (warp == 12) {
        tc::tmem_alloc(&sm.tmem, 512);
        tc::fence_before_sync();
    }
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem;
    if (warp < 8) {
        regs_inc<kRegsSoftmax>();
        softmax_rows<D, Q, FP8>(sm, p, u, kr, tmem, W, S, partial);
        __syncwarp();
        regs_dec<kRegs>();   // back to what the common code was compiled for
    } else if (warp < 12) {
        regs_dec<kRegsLoad>();
        load_tiles<D, Q, FP8>(sm, args, u, kr, S);
        __syncwarp();
        regs_inc<kRegs>();
    } else {
        regs_dec<kRegsMma>();
        if (warp == 12 && lane == 0) issue_products<D, Q>(sm, u, tmem, c.err);
        __syncwarp();
        regs_inc<kRegs>();
    }
    tc::fence_before_sync();
    if (partial) __threadfence();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 12) {
        if (sm.stop) {   // a wait gave up: let what was issued finish before the memory goes back
            if (lane == 0) {
                tc::commit(&sm.drain);
                mbar_wait_bounded(&sm.drain, 0, kLimitNs);
            }
            __syncwarp();
            tc::fence_after_sync();
        }
        tc::tmem_dealloc(tmem, 512);
    }
    if (!partial) return;
    // ---- the last of a unit's CTAs joins the pieces, in their order
    if (tid == 0) {
        const int done = atomicAdd(count, 1);
        sm.last = done == pieces - 1;
        if (sm.last) *count = 0;   // ready for the next call
        __threadfence();
    }
    __syncthreads();
    if (!sm.last || tid >= u.rows) return;
    const int r = u.r0 + tid;
    const float *at = ws.slot(blockIdx.x * splits, D) + tid;
    constexpr size_t step = SplitWs::slot_floats(D);
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < pieces; i++) m = fmaxf(m, __ldcg(at + i * step));
    const float base = m == -INFINITY ? 0.f : m;
    for (int i = 0; i < pieces; i++) l += ex2(__ldcg(at + i * step) - base) * __ldcg(at + i * step + kRowsCta);
    const float f = l == 0.f ? 0.f : (FP8 ? c.v_scale[p.layer * c.Hkv + u.h] : 1.f) / l;
    for (int d = 0; d < D; d += 32) {
        float o[32];
#pragma unroll
        for (int j = 0; j < 32; j++) o[j] = 0.f;
        for (int i = 0; i < pieces; i++) {
            const float a = ex2(__ldcg(at + i * step) - base);
#pragma unroll
            for (int j = 0; j < 32; j++) o[j] += a * __ldcg(at + i * step + (size_t)(2 + d + j) * kRowsCta);
        }
        store_row<Q>(p, u, r, d, o, f);
    }
    if (p.lse) p.lse[(size_t)(u.c0 + r / p.G) * p.Hq + u.h * p.G + r % p.G] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// The driver's tensor-map encoder, looked up once.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encoder()
{
    static const EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

cudaError_t encode(CUtensorMap *map, void *base, const PagedCache &c)
{
    const EncodeTiled fn = encoder();
    if (!fn) return cudaErrorSymbolNotFound;
    const cuuint64_t row = (cuuint64_t)c.D * 2;
    const cuuint64_t dims[3] = {(cuuint64_t)c.D, (cuuint64_t)c.Hkv * c.ps, (cuuint64_t)c.layers * c.pages};
    const cuuint64_t strides[2] = {row, row * c.Hkv * c.ps};
    const cuuint32_t box[3] = {64, (cuuint32_t)c.ps, 1}, step[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, typename Q, bool FP8>
cudaError_t launch_as(const AttnParams &p, cudaStream_t stream)
{
    static KernelSetup setup;
    constexpr size_t smem = sizeof(Smem<D>) + 1024;
    cudaError_t e = setup.get(kda_attn_prefill_kernel<D, Q, FP8>, kThreads, smem, 0, nullptr);
    if (e != cudaSuccess) return e;
    int sms = 0;
    if ((e = paged_sm_count(&sms)) != cudaSuccess) return e;
    // row tiles of all sequences: at most one partly filled tile each
    const long long by_total = (long long)p.total * p.G / kRowsCta + p.B;
    const long long by_len = (long long)p.B * (((long long)p.T * p.G + kRowsCta - 1) / kRowsCta);
    const long long tiles = by_total < by_len ? by_total : by_len, units = tiles * p.c.Hkv;
    if (units > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    // too few units to fill the SMs: split the keys
    const int most = sms < kMaxSplitCtas ? sms : kMaxSplitCtas;
    const int splits = units * 2 <= most ? (int)(most / units) : 1;
    Args a = {};
    a.p = p;
    if (!FP8 && ((e = encode(&a.k, p.c.k, p.c)) != cudaSuccess || (e = encode(&a.v, p.c.v, p.c)) != cudaSuccess)) return e;
    return launch_pdl(kda_attn_prefill_kernel<D, Q, FP8>, dim3((unsigned)units, (unsigned)splits), dim3(kThreads), smem, stream, a);
}

template <int D>
cudaError_t launch_types(const AttnParams &p, cudaStream_t stream)
{
    if (p.c.dtype == KDA_T_E4M3) return p.f16 ? launch_as<D, Half, true>(p, stream) : launch_as<D, Bf16, true>(p, stream);
    return p.f16 ? launch_as<D, Half, false>(p, stream) : launch_as<D, Bf16, false>(p, stream);
}

}  // namespace

size_t attn_prefill_workspace(int D) { return kMaxSplitCtas * sizeof(int) + kMaxSplitCtas * SplitWs::slot_floats(D) * sizeof(float); }

cudaError_t launch_attn_prefill(const AttnParams &p, cudaStream_t stream)
{
    return p.c.D == 128 ? launch_types<128>(p, stream) : launch_types<64>(p, stream);
}

}  // namespace kda
