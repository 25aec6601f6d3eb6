// kda_attn_prefill.cu -- attention of packed new tokens over a paged key-value cache
// (kda_attn_prefill), on the 5th-generation tensor cores.
//
// Mathematics.  The rows of one sequence and key head are its (token, query head) pairs in that
// order; a CTA takes 256 of them as two halves of 128 and walks the key tiles (128 keys) that its
// tokens see.  Per half and tile: S = Q K^T into tensor memory, one thread per row takes the row's
// maximum, P = exp2(S - m) back into tensor memory in 16 bits, O += P V with P as the tensor-memory
// operand.  The running maximum m is only moved (and O rescaled) when it grows by more than 2^8 (2^4 where P
// is half, see kShift): P stays in the range of its type, and l and O are FP32 sums of the same scale.
//
// Bound.  4 D flops for each visible (row, key) pair against D bytes moved once per 256 rows: the
// tensor cores, or the 128 x 128 exponentials of each tile next to them.  Two halves, so that one
// half's softmax runs while the tensor cores work on the other's products.
//
// Persistent: one CTA per SM takes (sequence, row tile, key head) units off a counter, the longest of a
// causal prompt first, so that one unit's queries and keys are on their way while the last one's sums are
// written (a CTA per unit spent 14 us of each unit outside its products).
//
// Roles: warps 0-3 and 4-7 are the softmax of the two halves (one thread per row), warps 8-11 copy
// keys and values into a ring of shared-memory tiles, warp 12 issues every MMA, warp 13 finds
// the next unit (14 and 15 only give their registers away; with a 4-bit cache 14 fetches codes).  Hand-over
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
// codes on their way.  Keys that are seen but whose table entry names no page come as zeros too, and the loaders
// leave the softmax a word for each tile that says which groups of 8 keys these are (4 x 4096 tokens 395.2 -> 397.7 us; with
// the pages looked up beside the sums 402 to 414).
//
// 4-bit caches: a code times its block's E4M3 scale is exact in a half (two significant bits by four, 2^-10 to 2688), so the tiles are
// halves, converted from 72 bytes a key of 128 dims.  Warp 14 brings whole pages' bytes by bulk copies and warps 8-11 only convert;
// bfloat16 queries come by TMA and are brought to halves in place by the softmax's threads.  4 x 4096 tokens, 32/8 heads: 516 us
// (16-bit caches 395).  As with E4M3 codes, the four warps looking up, fetching and converting, 824 us: a fetch took 1350 clocks
// beside a conversion of 650; with addresses once a tile 738; bulk copies 536.  Without the conversion's instructions 450: they
// share the issue slots and shared memory with the softmax, and neither waits long for the other.
#include <cuda.h>

#include "kda_attn_common.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kHalf = 128, kRowsCta = 256, kKeys = 128;
constexpr int kSoftmax = 256, kLoaders = 128, kThreads = kSoftmax + kLoaders + 128;
// Registers of a thread: all start with 128 (512 threads, the whole file), then the softmax holds a row
// of S at once; 256 x 184 + 128 x 80 + 128 x 64 = 65536.
constexpr int kRegs = 128, kRegsMma = 64;
constexpr int kRegsSoftmax = 184, kRegsLoad = 80;
constexpr int kHalfBytes = kKeys * 128;   // a tile's 64 head dims: 128 rows of 128 bytes
constexpr int kMaxSplitCtas = 256;             // CTAs of a launch, and pieces of split units
constexpr int kMinShare = 8;                   // key tiles of a piece at least
constexpr int kMaxSplits = 32;                 // pieces of a unit (their join reads one after the other)
constexpr uint64_t kLimitNs = 2000000000ull;   // bound of every wait
constexpr int kUnits = 2, kTable = 512;         // units on their way to the roles; sequences whose tile counts are kept on chip
constexpr int kGone = 8;                       // tiles whose missing pages are told to the softmax (four would do, see load_unit)

// What a CTA works on: rows [r0, r0 + rows) of the n * G of a sequence, and key tiles [ta, tb) of their range.
struct Unit {
    int idx;               // its number, -1: no more
    int row, h;            // cache row, key head
    int c0, n, len;        // first packed token, new tokens, row length
    int r0, rows, halves;
    int t0, g0;            // token and head of the group of row r0
    int p_first, p_last;   // positions of its first and last token
    int ta, tb, pieces;    // pieces > 1: the keys are split
    int slot, first, group;   // ... this piece's and the first one's place in the workspace, the split unit's number
};

// Bytes of a key: its elements or codes, and its block scales (E2M1).
template <int D, int KV>
struct KeyBytes {
    static constexpr int RB = KV == kKv16 ? D * 2 : KV == kKvE4M3 ? D : D / 2, SB = KV == kKvE2M1 ? D / 16 : 0;
};

// A ring of four tiles; with a cache of codes three, and three fetches of codes on their way to it.
template <int D, int KV>
struct Smem {
    static constexpr uint32_t kSlots = KV != kKv16 ? 3 : 4;
    static constexpr int kRaw = 3;
    uint8_t q[2][kHalf * D * 2];
    uint8_t kv[kSlots][kKeys * D * 2];
    uint8_t raw[KV != kKv16 ? kRaw : 1][KV != kKv16 ? kKeys * KeyBytes<D, KV>::RB : 16];
    uint8_t raw_scale[KV == kKvE2M1 ? kRaw : 1][KV == kKvE2M1 ? kKeys * KeyBytes<D, KV>::SB : 16];
    uint64_t raw_full[kRaw], raw_empty[kRaw], q_raw;   // E2M1: raw items, and queries, of warp 14
    uint64_t q_full[2], q_empty, full[kSlots], empty[kSlots], s_full[2], p_full[2], o_full[2], u_full[kUnits], u_empty[kUnits], join, drain;
    unsigned gone[kGone];                   // by the tile's number: groups of 8 keys that are seen but have no page
    Unit unit[kUnits];
    int before[kTable + 1], warp_sum[16];   // row tiles of the sequences before each one
    int4 seq[kTable];                       // row, length, new tokens, first packed token
    float q_scale[2][kRowsCta];             // E4M3 cache: what a unit's scores have to be multiplied with, by its parity
    uint32_t tmem;
    int last;
    volatile int stop;
};

struct Args {
    AttnParams p;
    CUtensorMap k, v;   // [layers pages][Hkv page_size][D], boxes of one page's tokens x 64 head dims
    CUtensorMap q;      // [tokens][heads][D], boxes of 128 rows (token, head of the group) x 64 head dims
    bool q_map;         // ... which need a group that divides 128 (see map_queries)
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

__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1)
{
    asm("{\n\t.reg .b64 a, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 d, {%0, %1};\n\tadd.rn.f32x2 d, d, a;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1));
}

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

// Bounded wait: after two seconds, or when another role has given up, the CTA winds down.
template <typename SM>
__device__ __forceinline__ bool wait_long(SM &sm, uint64_t *bar, uint32_t parity, int *err)
{
    const uint64_t t0 = globaltimer_ns();
    while (!sm.stop) {
        for (int i = 0; i < 64; i++)
            if (mbar_try_wait(bar, parity)) return true;
        if (globaltimer_ns() - t0 > kLimitNs) {
            sm.stop = 1;
            atomicOr(err, KDA_DEVERR_TIMEOUT);
        }
    }
    return false;
}
// ... by all lanes of a warp, which agree on the outcome
template <typename SM>
__device__ __forceinline__ bool wait_warp(SM &sm, uint64_t *bar, uint32_t parity, int *err)
{
    for (int i = 0; i < 64; i++)   // the usual wait ends here, without a look at the clock
        if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
    return __all_sync(~0u, wait_long(sm, bar, parity, err));
}

// A role's k-th unit, left by warp 13 in shared memory: null when there is no more (or a wait gave up).
template <typename SM>
__device__ __forceinline__ const Unit *unit_of(SM &sm, int k, int *err)
{
    if (!wait_warp(sm, &sm.u_full[k % kUnits], (k / kUnits) & 1, err)) return nullptr;
    const Unit *u = &sm.unit[k % kUnits];
    return u->idx >= 0 ? u : nullptr;
}
// ... and that this warp is done with it.
template <typename SM>
__device__ __forceinline__ void unit_done(SM &sm, int k)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.u_empty[k % kUnits]);
}

// True in one lane, the same one at every call.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ---- warp 12: products, in the order that lets one half's softmax run beside the other's products: P V of
// a tile, then Q K^T of the half's next one (which overwrites P only after it is read: one thread's products
// run in order).  The whole warp walks the loop, so that the descriptors stay in uniform registers, and
// one lane issues.
// `item`: ring items so far; `tiles`: key tiles so far of each half; `units`: units with products so far
template <int D, typename Q, int HALVES, typename SM>
__device__ __forceinline__ bool issue_products(SM &sm, int n, uint32_t tmem, uint32_t &item, uint32_t *tiles, uint32_t &units, int *err)
{
    const uint64_t q_desc = desc_sw128(smem_u32(sm.q[0]), 16u), k_desc = desc_sw128(smem_u32(sm.kv[0]), 16u),
                   v_desc = desc_sw128(smem_u32(sm.kv[0]), kHalfBytes);
    constexpr uint32_t kSlots = SM::kSlots, kTile = kKeys * D * 2 >> 4;   // a ring slot, a half's queries, in descriptor units
    auto slot_wait = [&](uint32_t it) { return wait_warp(sm, &sm.full[it % kSlots], (it / kSlots) & 1, err); };
    auto qk = [&](int h, uint32_t it, bool last_tile) {
        const uint64_t ad = q_desc + h * kTile, bd = k_desc + (it % kSlots) * kTile;
        if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; k++) {   // 16 head dims: 32 bytes further in the half's rows
                const uint32_t step = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
                tc::mma(tmem + Cols<D>::s(h), ad + step, bd + step, idesc<Q>(kKeys), k > 0);
            }
            tc::commit(&sm.s_full[h]);
            if (h + 1 == HALVES) {
                tc::commit(&sm.empty[it % kSlots]);
                if (last_tile) tc::commit(&sm.q_empty);
            }
        }
    };
    if (!wait_warp(sm, &sm.q_full[units & 1], (units >> 1) & 1, err)) return false;
    if (!slot_wait(item)) return false;
    tc::fence_after_sync();
#pragma unroll
    for (int h = 0; h < HALVES; h++) qk(h, item, n == 1);
    for (int i = 0; i < n; i++) {
        const uint32_t it = item + 2 * i + 1;
        if (!slot_wait(it)) return false;
        const bool more = i + 1 < n;
        if (more && !slot_wait(it + 1)) return false;
#pragma unroll
        for (int h = 0; h < HALVES; h++) {
            const uint64_t bd = v_desc + (it % kSlots) * kTile;
            if (!wait_warp(sm, &sm.p_full[h], (tiles[h] + i) & 1, err)) return false;
            tc::fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; k++)   // 16 keys: two groups of 8 rows
                    mma_ts(tmem + Cols<D>::o(h), tmem + Cols<D>::p(h) + 8 * k, bd + k * (2048u >> 4), idesc<Q>(D) | (1u << 16), i > 0 || k > 0);
                if (!more) tc::commit(&sm.o_full[h]);
                if (h + 1 == HALVES) tc::commit(&sm.empty[it % kSlots]);
            }
            if (more) qk(h, it + 1, i + 2 == n);
        }
    }
    item += 2 * n;
    units++;
#pragma unroll
    for (int h = 0; h < HALVES; h++) tiles[h] += n;
    return true;
}

template <int D, typename Q, typename SM>
__device__ void mma_role(SM &sm, uint32_t tmem, int *err)
{
    uint32_t item = 0, tiles[2] = {0, 0}, units = 0;
    for (int k = 0; const Unit *u = unit_of(sm, k, err); k++) {
        // (the reductions leave their results in uniform registers)
        const int n = __reduce_max_sync(~0u, u->tb - u->ta);
        const bool two = __all_sync(~0u, u->halves == 2);
        unit_done(sm, k);
        if (n == 0) continue;
        if (!(two ? issue_products<D, Q, 2>(sm, n, tmem, item, tiles, units, err)
                                             : issue_products<D, Q, 1>(sm, n, tmem, item, tiles, units, err)))
            return;
    }
}

// Token (of the unit's sequence) and index in [token, head] of a unit's row x.  The quotient comes from the
// reciprocal: (g0 + x + 1/2) / G is at least 1 / (2 G) from a whole number, far more than the product's error.
__device__ __forceinline__ int row_token(const AttnParams &p, const Unit &u, int x) { return u.t0 + (int)((u.g0 + x + 0.5f) * p.inv_g); }
__device__ __forceinline__ size_t row_index(const AttnParams &p, const Unit &u, int x)
{
    const int t = row_token(p, u, x);
    return (size_t)(u.c0 + t) * p.Hq + u.h * p.G + (u.r0 + x - t * p.G);
}

// Whether bfloat16 queries come as they are (by warp 14, 4-bit cache) and are brought to halves in place by the softmax's threads.
template <typename Q, int KV>
__device__ __forceinline__ bool queries_in_place(const Args &args) { return KV == kKvE2M1 && !Q::is_half && args.q_map; }

// ---- warps 8-11: a unit's queries, then keys and values of tile i as ring items 2 i and 2 i + 1
// (`item`: ring items so far, `units`: units so far)
template <int D, typename Q, int KV>
__device__ bool load_unit(Smem<D, KV> &sm, const Args &args, const Unit &u, int W, int S, uint32_t &item, uint32_t &units)
{
    using SM = Smem<D, KV>;
    const AttnParams &p = args.p;
    constexpr uint32_t kSlots = SM::kSlots;
    const KeyRange<kKeys> kr(u.p_first, u.p_last, u.len, W, S);
    const PagedCache &c = p.c;
    const int tid = threadIdx.x - kSoftmax, w = tid >> 5, lane = tid & 31, r8 = lane & 7, q4 = lane >> 3;
    const int n = u.tb - u.ta;
    constexpr bool CODES = KV != kKv16;
    constexpr int RB = KeyBytes<D, KV>::RB, SB = KeyBytes<D, KV>::SB;
    constexpr int CPR = RB / 16;              // 16-byte chunks of a key
    constexpr int PASS = CPR / 4;             // passes of four chunks over a group of 8 keys
    constexpr int GR = kKeys / 8 / 4;         // groups of 8 keys of a warp: w, w + 4, ...
    const size_t head_bytes = (size_t)c.ps * (RB + SB);
    // page of key group `lane` (16 groups of a tile), 0 where none of its keys is seen (and no page is looked at)
    auto pages_of = [&](int i) {
        const int k0 = kr.tile(u.ta + i) * kKeys + lane * 8;
        if (i >= n || lane >= kKeys / 8 || k0 >= kr.end || !(k0 + 8 > kr.lo || k0 < S)) return 0;
        return __ldg(c.table + (size_t)u.row * c.width + (k0 >> c.ps_log2));
    };
    int pages = 0, pages_next = 0;
    if constexpr (KV != kKvE2M1) pages = pages_of(0), pages_next = pages_of(1);
    // Which groups are seen but have no page, for the softmax: written ahead of this thread's arrival for the tile's keys,
    // which their products wait for.  The word of the tile four before has been read by then: an item written now (or
    // sent three items ahead, E4M3) has waited for the keys of the tile three before it at least, whose products
    // are only issued when the softmax has handed over the tile before them.
    [[maybe_unused]] auto tell_gone = [&](uint32_t ring) {
        const unsigned gone = __ballot_sync(~0u, (unsigned)pages >= (unsigned)c.pages);
        if (tid == 0 && !(ring & 1)) sm.gone[(ring >> 1) % kGone] = gone;
        return gone;
    };
    // queries; without a map 16 (or 8) lanes for a row, zeros past the unit's rows (the copies of 64 KiB by
    // threads took 11000 clocks, longer than the sums they are to overlap)
    auto load_queries = [&]() {
        if (units > 0 && !wait_warp(sm, &sm.q_empty, (units - 1) & 1, c.err)) return false;
        if constexpr (CODES && !Q::is_half) {   // through registers, as halves
            constexpr int LPR = D / 8, STEP = kLoaders / LPR;
            const int g = tid % LPR;
            const uint16_t *base = p.q + (long long)u.c0 * p.ql.token + (long long)(u.h * p.G) * p.ql.head + g * 8;
#pragma unroll 4
            for (int i = 0; i < 2 * kHalf / STEP; i++) {
                const int r = i * STEP + tid / LPR;
                if (i * STEP >= u.halves * kHalf) break;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (r < u.rows) {
                    const int t = row_token(p, u, r);
                    x = __ldg(reinterpret_cast<const uint4 *>(base + t * p.ql.token + (u.r0 + r - t * p.G) * p.ql.head));
                }
                uint32_t mag = max_magnitude(0, x);
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1) mag = max(mag, __shfl_xor_sync(~0u, mag, o));
                float down, up;
                query_scale(mag, down, up);
                *reinterpret_cast<uint4 *>(sm.q[0] + (r >> 7) * (kHalf * D * 2) + chunk_at(r & 127, g)) = scaled_halves(x, down);
                if (g == 0) sm.q_scale[units & 1][r] = up;
            }
            return true;
        }
        if (args.q_map) {   // by TMA; rows past the unit's are other tokens' (or zeros), and what comes of them is not stored
            if (tid == 0) mbar_arrive_expect_tx(&sm.q_full[units & 1], u.halves * (kHalf * D * 2));
            else mbar_arrive(&sm.q_full[units & 1]);
            __syncwarp();
            if (tid < u.halves * (D / 64)) {
                const int hf = tid / (D / 64), x = tid % (D / 64);
                tma_load_3d(smem_u32(sm.q[0]) + hf * (kHalf * D * 2) + x * kHalfBytes, &args.q, x * 64, u.h * p.G,
                            u.c0 + (u.r0 + hf * kHalf) / p.G, &sm.q_full[units & 1]);
            }
            return true;
        }
        constexpr int LPR = D / 8, STEP = kLoaders / LPR;   // lanes of a row, rows of a pass
        const int g = tid % LPR, step_t = STEP / p.G, step_q = STEP - step_t * p.G;
        int r = tid / LPR, t = (u.r0 + r) / p.G, q = u.r0 + r - t * p.G;   // the row's token and head of the group
        const uint16_t *base = p.q + (long long)u.c0 * p.ql.token + (long long)(u.h * p.G) * p.ql.head + g * 8;
#pragma unroll 2
        for (int i = 0; i < 2 * kHalf / STEP; i++) {
            if (r < u.halves * kHalf) {
                const bool live = r < u.rows;
                cp_async16(sm.q[0] + (r >> 7) * (kHalf * D * 2) + chunk_at(r & 127, g),
                           live ? base + t * p.ql.token + q * p.ql.head : p.q, live ? 16 : 0);
            }
            r += STEP;
            t += step_t;
            q += step_q;
            if (q >= p.G) q -= p.G, t++;
        }
        return true;
    };
    auto queries_done = [&]() {
        if (args.q_map && !(CODES && !Q::is_half)) return;
        cp_async_wait_all();
        tc::fence_smem_to_async();
        mbar_arrive(&sm.q_full[units & 1]);
    };
    // source of this lane's key of group gi of tile i; null where nothing is read
    [[maybe_unused]] auto source = [&](const uint8_t *base, int i, int gi, int pg) -> const uint8_t * {
        const int k0 = kr.tile(u.ta + i) * kKeys + gi * 8, j = k0 + r8;
        if (!(j < kr.end && (j >= kr.lo || j < S))) return nullptr;
        if ((unsigned)pg >= (unsigned)c.pages) {
            atomicOr(c.err, KDA_DEVERR_PAGE);
            return nullptr;
        }
        return base + (((size_t)p.layer * c.pages + pg) * c.Hkv + u.h) * head_bytes + (size_t)(j & (c.ps - 1)) * RB;
    };
    if constexpr (!CODES) {
        for (int it = 0; it < 2 * n; it++) {
            const uint32_t ring = item + it;
            const int i = it >> 1, slot = ring % kSlots, k0 = kr.tile(u.ta + i) * kKeys;
            const uint8_t *base = it & 1 ? c.v : c.k;
            if (ring >= kSlots && !wait_warp(sm, &sm.empty[slot], (ring / kSlots - 1) & 1, c.err)) return false;
            // every key is seen by some token and has a page (the four warps hold the same page ids)
            const bool whole = tell_gone(ring) == 0 && k0 + kKeys <= kr.end && (k0 >= kr.lo || k0 + kKeys <= S);
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
            if (it == 0 && !load_queries()) return false;
            if (it == 1) queries_done();   // the first keys and values were on their way meanwhile
            if (it & 1) {
                pages = pages_next;
                pages_next = pages_of(i + 2);
            }
        }
    } else if constexpr (KV == kKvE2M1) {
        // Warp 14 fetches the codes (fetch_unit); these warps only convert them, 32 keys each.  (Two warps for keys and two for
        // values, with twice the items on their way: 620 us against 510; a ring of four tiles with two or three fetches
        // ahead, or three tiles with five: within 2 % or slower.)
        constexpr int ROWS = 32 / CPR;   // a pass: chunk cp of ROWS keys
        const int row = lane % ROWS, cp = lane / ROWS, at_codes = (w * 32 + row) * RB + cp * 16, at_scales = (w * 32 + row) * SB + 2 * cp;
        int at_tile[4];   // (the rows of later passes are whole groups of 8 further: the same places in their swizzle)
#pragma unroll
        for (int y = 0; y < 4; y++) at_tile[y] = chunk_at(w * 32 + row, cp * 4 + y);
        for (int it = 0; it < 2 * n; it++) {
            const uint32_t ring = item + it;
            const int slot = ring % kSlots, from = ring % SM::kRaw;
            if (!wait_warp(sm, &sm.raw_full[from], (ring / SM::kRaw) & 1, c.err)) return false;
            if (ring >= kSlots && !wait_warp(sm, &sm.empty[slot], (ring / kSlots - 1) & 1, c.err)) return false;
            const uint8_t *src = sm.raw[from] + at_codes, *sc = sm.raw_scale[from] + at_scales;
#pragma unroll
            for (int a = 0; a < CPR; a++) {   // 32 codes, two blocks: exact in halves
                const uint4 v = *reinterpret_cast<const uint4 *>(src + a * ROWS * RB);
                const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
                const uint32_t s2 = e4m3x2_half2(*reinterpret_cast<const uint16_t *>(sc + a * ROWS * SB));
                const uint32_t s[2] = {__byte_perm(s2, s2, 0x1010), __byte_perm(s2, s2, 0x3232)};
#pragma unroll
                for (int y = 0; y < 4; y++) {
                    uint32_t e[4];
                    e2m1x8_half8(ws[y], e);
                    *reinterpret_cast<uint4 *>(sm.kv[slot] + at_tile[y] + a * ROWS * 128) =
                        make_uint4(hmul2(e[0], s[y >> 1]), hmul2(e[1], s[y >> 1]), hmul2(e[2], s[y >> 1]), hmul2(e[3], s[y >> 1]));
                }
            }
            tc::fence_smem_to_async();
            mbar_arrive(&sm.full[slot]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.raw_empty[from]);
            // the first keys were converted while the last unit's queries were still in use (softmax_role converts queries that come by TMA)
            if (it == 0 && !queries_in_place<Q, KV>(args)) {
                if (!load_queries()) return false;
                queries_done();
            }
        }
    } else {
        if (!load_queries()) return false;
        queries_done();
        // Codes come to shared memory three items ahead (each thread's own pieces, so that only its own copies are
        // waited for) and are converted (exactly) to halves on their way into the ring.  With one item ahead,
        // in registers, a tile pair took 3.0 us; like this 2.5 us (16-bit caches: 1.54; both with half queries).  4 x 4096 tokens,
        // 32/8 heads: 566 us with half queries, 808 with bfloat16 ones, which come through these warps' registers.
        constexpr int kRaw = Smem<D, KV>::kRaw;
        int sent = 0;   // items whose copies are under way
        auto send = [&]() {
            if (sent < 2 * n) {
                tell_gone(item + sent);
                const uint8_t *base = sent & 1 ? c.v : c.k;
                uint8_t *dst = sm.raw[sent % kRaw] + tid * 16;
#pragma unroll
                for (int a = 0; a < GR; a++) {
                    const int gi = w + 4 * a;
                    const uint8_t *src = source(base, sent >> 1, gi, __shfl_sync(~0u, pages, gi));
#pragma unroll
                    for (int x = 0; x < PASS; x++)
                        cp_async16(dst + (a * PASS + x) * (kLoaders * 16), src ? src + (x * 4 + q4) * 16 : c.k, src ? 16 : 0);
                }
                if (sent & 1) {
                    pages = pages_next;
                    pages_next = pages_of((sent >> 1) + 2);
                }
            }
            sent++;
            cp_async_commit();
        };
        for (int i = 0; i < kRaw; i++) send();
        for (int it = 0; it < 2 * n; it++) {
            const uint32_t ring = item + it;
            const int slot = ring % kSlots;
            cp_async_wait<kRaw - 1>();
            if (ring >= kSlots && !wait_warp(sm, &sm.empty[slot], (ring / kSlots - 1) & 1, c.err)) return false;
            const uint4 *src = reinterpret_cast<const uint4 *>(sm.raw[it % kRaw]) + tid;
#pragma unroll
            for (int a = 0; a < GR; a++)
#pragma unroll
                for (int x = 0; x < PASS; x++) {
                    const uint4 v = src[(a * PASS + x) * kLoaders];
                    const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
                    uint32_t e[8];
#pragma unroll
                    for (int s = 0; s < 4; s++) e4m3x4_half4(ws[s], e[2 * s], e[2 * s + 1]);
#pragma unroll
                    for (int s = 0; s < 2; s++)
                        *reinterpret_cast<uint4 *>(sm.kv[slot] + chunk_at((w + 4 * a) * 8 + r8, (x * 4 + q4) * 2 + s)) =
                            make_uint4(e[4 * s], e[4 * s + 1], e[4 * s + 2], e[4 * s + 3]);
                }
            tc::fence_smem_to_async();
            mbar_arrive(&sm.full[slot]);
            send();
        }
        cp_async_wait<0>();
    }
    item += 2 * n;
    units++;
    return true;
}

// ---- warp 14, 4-bit cache: a unit's codes and block scales as they are (raw items 2 i and 2 i + 1 of tile i), whole pages by bulk
// copies, and its bfloat16 queries
template <int D, typename Q>
__device__ bool fetch_unit(Smem<D, kKvE2M1> &sm, const Args &args, const Unit &u, int W, int S, uint32_t &item, uint32_t &units, uint32_t &written)
{
    using SM = Smem<D, kKvE2M1>;
    constexpr int RB = KeyBytes<D, kKvE2M1>::RB, SB = KeyBytes<D, kKvE2M1>::SB, CPR = RB / 16, ROWS = 32 / CPR;
    const AttnParams &p = args.p;
    const PagedCache &c = p.c;
    const int lane = threadIdx.x & 31, n = u.tb - u.ta;
    const KeyRange<kKeys> kr(u.p_first, u.p_last, u.len, W, S);
    const uint32_t page_bytes = (uint32_t)c.page_bytes();   // under 2^27
    const size_t head_bytes = (size_t)c.ps * (RB + SB);
    const uint8_t *k_head = c.k + ((size_t)p.layer * c.pages * c.Hkv + u.h) * head_bytes;
    const ptrdiff_t v_minus_k = c.v - c.k;
    // page of key group `lane` (16 groups of a tile), 0 where none of its keys is seen (and no page is looked at)
    auto pages_of = [&](int i) {
        const int k0 = kr.tile(u.ta + i) * kKeys + lane * 8;
        if (i >= n || lane >= kKeys / 8 || k0 >= kr.end || !(k0 + 8 > kr.lo || k0 < S)) return 0;
        return __ldg(c.table + (size_t)u.row * c.width + (k0 >> c.ps_log2));
    };
    int pages = pages_of(0), pages_next = pages_of(1);
    for (int i = 0; i < n; i++) {
        const int k0 = kr.tile(u.ta + i) * kKeys;
        const unsigned gone = __ballot_sync(~0u, (unsigned)pages >= (unsigned)c.pages);
        const bool whole = gone == 0 && k0 + kKeys <= kr.end && (k0 >= kr.lo || k0 + kKeys <= S);
        // lane x: page x of the tile
        const int tile_pages = kKeys >> c.ps_log2 ? kKeys >> c.ps_log2 : 1, page = __shfl_sync(~0u, pages, (lane << (c.ps_log2 - 3)) & 31);
        const uint8_t *head = k_head + (size_t)(uint32_t)page * page_bytes;
        for (int kv = 0; kv < 2; kv++) {
            const uint32_t ring = item + 2 * i + kv;
            const int to = ring % SM::kRaw;
            uint64_t *bar = &sm.raw_full[to];
            const ptrdiff_t add = kv ? v_minus_k : 0;
            if (ring >= SM::kRaw && !wait_warp(sm, &sm.raw_empty[to], (ring / SM::kRaw - 1) & 1, c.err)) return false;
            // (told ahead of the tile's keys, see tell_gone: its raw item has waited for the conversion of the one kRaw items before;
            // the plain arrival releases the word, which an arrival by asynchronous copies does not)
            if (lane == 0) {
                if (kv == 0) sm.gone[(ring >> 1) % kGone] = gone;
                mbar_arrive(bar);
            }
            if (whole) {
                if (written >> to & 1) {   // before a bulk copy overwrites what these lanes' copies wrote
                    tc::fence_smem_to_async();
                    written &= ~(1u << to);
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive_expect_tx(bar, kKeys * (RB + SB));
                else mbar_arrive(bar);
                __syncwarp();
                if (lane < tile_pages) {
                    const uint32_t codes = (uint32_t)(RB << c.ps_log2), scales = (uint32_t)(SB << c.ps_log2);
                    bulk_load(sm.raw[to] + lane * codes, head + add, codes, bar);
                    bulk_load(sm.raw_scale[to] + lane * scales, head + add + codes, scales, bar);
                }
            } else {   // zeros for the keys that no token sees, or that have no page
                auto key = [&](int r) -> const uint8_t * {   // head of its page, null: zeros
                    const int j = k0 + r, pg = __shfl_sync(~0u, pages, r >> 3);
                    if (!(j < kr.end && (j >= kr.lo || j < S))) return nullptr;
                    if ((unsigned)pg >= (unsigned)c.pages) {
                        atomicOr(c.err, KDA_DEVERR_PAGE);
                        return nullptr;
                    }
                    return k_head + (size_t)(uint32_t)pg * page_bytes + add;
                };
                for (int r = lane % ROWS; r < kKeys; r += ROWS) {
                    const uint8_t *h = key(r);
                    cp_async16(sm.raw[to] + r * RB + lane / ROWS * 16, h ? h + ((k0 + r) & (c.ps - 1)) * RB + lane / ROWS * 16 : c.k, h ? 16 : 0);
                }
                for (int r = lane; r < kKeys; r += 32) {
                    const uint8_t *h = key(r);
                    cp_async_small<SB>(smem_u32(sm.raw_scale[to] + r * SB), h ? h + (size_t)c.ps * RB + ((k0 + r) & (c.ps - 1)) * SB : c.k, h ? SB : 0);
                }
                written |= 1u << to;
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
            }
            if constexpr (!Q::is_half)
                if (i == 0 && kv == 0 && queries_in_place<Q, kKvE2M1>(args)) {   // rows past the unit's are other tokens' (or zeros), and what comes of them is not stored
                    if (units > 0 && !wait_warp(sm, &sm.q_empty, (units - 1) & 1, c.err)) return false;
                    if (lane == 0) mbar_arrive_expect_tx(&sm.q_raw, u.halves * (kHalf * D * 2));
                    __syncwarp();
                    if (lane < u.halves * (D / 64)) {
                        const int hf = lane / (D / 64), x = lane % (D / 64);
                        tma_load_3d(smem_u32(sm.q[0]) + hf * (kHalf * D * 2) + x * kHalfBytes, &args.q, x * 64, u.h * p.G,
                                    u.c0 + (u.r0 + hf * kHalf) / p.G, &sm.q_raw);
                    }
                }
        }
        pages = pages_next;
        pages_next = pages_of(i + 2);
    }
    item += 2 * n;
    units++;
    return true;
}

template <int D, typename Q, int KV>
__device__ void fetch_role(Smem<D, KV> &sm, const Args &args, int W, int S)
{
    if constexpr (KV == kKvE2M1) {
        uint32_t item = 0, units = 0, written = 0;
        for (int k = 0; const Unit *at = unit_of(sm, k, args.p.c.err); k++) {
            const Unit u = *at;
            unit_done(sm, k);
            if (u.tb > u.ta && !fetch_unit<D, Q>(sm, args, u, W, S, item, units, written)) break;
        }
        cp_async_wait<0>();
        // where a wait gave up, copies may still be landing: let them
        if (sm.stop) {
            for (int i = 0; i < Smem<D, KV>::kRaw; i++)
                for (uint32_t parity = 0; parity < 2; parity++) mbar_wait_bounded(&sm.raw_full[i], parity, kLimitNs / 16);
            for (uint32_t parity = 0; parity < 2; parity++) mbar_wait_bounded(&sm.q_raw, parity, kLimitNs / 16);
        }
    }
}

template <int D, typename Q, int KV>
__device__ void load_role(Smem<D, KV> &sm, const Args &args, int W, int S)
{
    constexpr uint32_t kSlots = Smem<D, KV>::kSlots;
    uint32_t item = 0, units = 0;
    for (int k = 0; const Unit *at = unit_of(sm, k, args.p.c.err); k++) {
        const Unit u = *at;
        unit_done(sm, k);
        if (u.tb > u.ta && !load_unit<D, Q, KV>(sm, args, u, W, S, item, units)) break;
    }
    cp_async_wait<0>();
    // where a wait gave up, tiles may still be landing: let them (the last one of each slot)
    if (sm.stop)
        for (uint32_t i = item < kSlots ? 0 : item - kSlots; i < item + kSlots; i++)
            mbar_wait_bounded(&sm.full[i % kSlots], (i / kSlots) & 1, kLimitNs / 8);
}

struct SplitWs {   // partial results of split units: (m, l) and O by column, so that threads (rows) are contiguous
    float *data;
    static constexpr size_t slot_floats(int D) { return (size_t)kRowsCta * (D + 2); }
    __device__ float *slot(int s, int D) const { return data + (size_t)s * slot_floats(D); }
};

// 32 outputs of a row.  A warp's rows are apart, so each store instruction goes to 32 lines: whole 32-byte
// sectors where the output's alignment allows it, which halves their number.
template <typename Q>
__device__ __forceinline__ void store_row(uint16_t *dst, bool wide, const float *o, float f)
{
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; i++) w[i] = Q::pack(o[2 * i] * f, o[2 * i + 1] * f);
    if (wide) {
#pragma unroll
        for (int i = 0; i < 2; i++)
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                         ::"l"(dst + 16 * i), "r"(w[8 * i]), "r"(w[8 * i + 1]), "r"(w[8 * i + 2]), "r"(w[8 * i + 3]),
                           "r"(w[8 * i + 4]), "r"(w[8 * i + 5]), "r"(w[8 * i + 6]), "r"(w[8 * i + 7]) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) reinterpret_cast<uint4 *>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}
__device__ __forceinline__ bool wide_stores(const AttnParams &p) { return (reinterpret_cast<uintptr_t>(p.out) & 31) == 0; }

// One row of a split unit from its pieces; `at`: the first piece's m of this row
template <int D, typename Q, int KV>
__device__ __noinline__ void join_row(const AttnParams &p, const Unit &u, const float *at)
{
    const size_t row = row_index(p, u, threadIdx.x);
    uint16_t *dst = p.out + row * D;
    constexpr size_t step = SplitWs::slot_floats(D);
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < u.pieces; i++) m = fmaxf(m, __ldcg(at + i * step));
    const float base = m == -INFINITY ? 0.f : m;
    for (int i = 0; i < u.pieces; i++) l += ex2(__ldcg(at + i * step) - base) * __ldcg(at + i * step + kRowsCta);
    const float f = l == 0.f ? 0.f : (KV != kKv16 ? p.c.v_scale[p.layer * p.c.Hkv + u.h] : 1.f) / l;
    for (int d = 0; d < D; d += 32) {
        float o[32];
#pragma unroll
        for (int j = 0; j < 32; j++) o[j] = 0.f;
        for (int i = 0; i < u.pieces; i++) {
            const float a = ex2(__ldcg(at + i * step) - base);
#pragma unroll
            for (int j = 0; j < 32; j++) o[j] += a * __ldcg(at + i * step + (size_t)(2 + d + j) * kRowsCta);
        }
        store_row<Q>(dst + d, wide_stores(p), o, f);
    }
    if (p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---- warps 0-7: one thread per row (`tiles`, `units`: this half's key tiles and units so far; `all_units`:
// those of either half, `all_tiles`: their key tiles)
template <int D, typename Q, int KV>
__device__ bool softmax_unit(Smem<D, KV> &sm, const AttnParams &p, const Unit &u, uint32_t tmem, int W, int S, bool in_place, float q_up, float *partial,
                             uint32_t &tiles, uint32_t &units, uint32_t all_units, uint32_t all_tiles)
{
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, h = tid >> 7, rl = tid & 127, w = tid >> 5;
    const int n = u.tb - u.ta;
    constexpr bool CODES = KV != kKv16;
    const KeyRange<kKeys> kr(u.p_first, u.p_last, u.len, W, S);
    const int x = h * kHalf + rl;                                // row of the unit
    const bool live = x < u.rows;
    using P = std::conditional_t<CODES, Half, Q>;                  // type of the products
    float row_scale = 1.f;
    if constexpr (CODES && !Q::is_half) {
        if (in_place) row_scale = q_up;
        else {
            // (the barrier of this parity cannot move on again before this half's last scores of the unit are read)
            if (!wait_warp(sm, &sm.q_full[all_units & 1], (all_units >> 1) & 1, c.err)) return false;
            row_scale = sm.q_scale[all_units & 1][x];
        }
    }
    const float sc = score_scale(p.scale_log2 * (CODES ? c.k_scale[p.layer * c.Hkv + u.h] : 1.f) * row_scale);
    const int first = u.len - u.n;
    const int pos = first + row_token(p, u, min(x, u.rows - 1));  // this row's position
    const int lo = (int)max(-0x7fffffffll, (long long)pos - W + 1);
    // positions of the half's first and last row: whether a tile is seen by all of it
    const int p_lo = first + row_token(p, u, h * kHalf), p_hi = first + row_token(p, u, min(h * kHalf + kHalf, u.rows) - 1);
    const long long lo_all = (long long)p_hi - W + 1;
    const uint32_t lane_base = tmem + ((uint32_t)(w & 3) * 32u << 16);
    const uint32_t ts = lane_base + Cols<D>::s(h), tp = lane_base + Cols<D>::p(h), to = lane_base + Cols<D>::o(h);
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < n; i++) {
        const int k0 = kr.tile(u.ta + i) * kKeys;
        const bool all = k0 + kKeys - 1 <= p_lo && (k0 >= lo_all || k0 + kKeys <= S);
        if (!wait_warp(sm, &sm.s_full[h], (tiles + i) & 1, c.err)) return false;
        tc::fence_after_sync();
        uint32_t v[kKeys];
#pragma unroll
        for (int q = 0; q < 4; q++) tmem_ld32_async(ts + 32 * q, v + 32 * q);
        uint32_t gone;   // on its way beside them
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(gone) : "r"(smem_u32(&sm.gone[(all_tiles + i) % kGone])) : "memory");
#pragma unroll
        for (int q = 0; q < 4; q++) tmem_wait_ld(v + 32 * q);
        if (!all || gone) {
            const int hi_j = pos - k0, lo_j = max(lo, k0) - k0, s_j = S - k0;
#pragma unroll
            for (int j = 0; j < kKeys; j++)
                if (!(j <= hi_j && (j >= lo_j || j < s_j))) v[j] = 0xff800000u;   // -inf
            if (gone) {
#pragma unroll
                for (int j = 0; j < kKeys; j++)
                    if (gone >> (j >> 3) & 1) v[j] = 0xff800000u;
            }
        }
        float mx8[8];
#pragma unroll
        for (int j = 0; j < 8; j++) mx8[j] = fmaxf(__uint_as_float(v[j]), __uint_as_float(v[j + 8]));
#pragma unroll
        for (int j = 16; j < kKeys; j += 16)
#pragma unroll
            for (int x = 0; x < 8; x++) mx8[x] = fmaxf(fmaxf(mx8[x], __uint_as_float(v[j + x])), __uint_as_float(v[j + 8 + x]));
        const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])), fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        const float m_new = fmaxf(m, P::kShift != 0.f ? fmaf(mx, sc, -P::kShift) : mx * sc);   // (m: kShift below the maximum)
        if (i == 0) m = m_new;
        else if (__any_sync(~0u, m_new > m + P::kGrow)) {
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
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int q = 0; q < 2; q++) {
#pragma unroll
            for (int j = 32 * q; j < 32 * q + 32; j++) {
                float e0, e1;
                tc::fma2(e0, e1, __uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]), sc, sc, -base, -base);
                e0 = ex2(e0), e1 = ex2(e1);
                if (j & 1) add2(s2, s3, e0, e1);
                else add2(s0, s1, e0, e1);
                v[j] = P::pack(e0, e1);   // rounded to 16 bits for the product; l sums it unrounded
            }
            tmem_st32(tp + 32 * q, v + 32 * q);
        }
        l += (s0 + s2) + (s1 + s3);
        tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(&sm.p_full[h]);
    }
    if (!wait_warp(sm, &sm.o_full[h], units & 1, c.err)) return false;
    tc::fence_after_sync();
    tiles += n;
    units++;
    const float f = l == 0.f ? 0.f : (CODES ? c.v_scale[p.layer * c.Hkv + u.h] : 1.f) / l;
    const size_t row = row_index(p, u, x);
    uint16_t *dst = p.out + row * D;
    const bool wide = wide_stores(p);
#pragma unroll 1
    for (int q = 0; q < D / 32; q++) {
        uint32_t v[32];
        tmem_ld32(to + 32 * q, v);
        if (partial) {
#pragma unroll
            for (int j = 0; j < 32; j++) __stcg(partial + (2 + 32 * q + j) * kRowsCta + tid, __uint_as_float(v[j]));
        } else if (live) {
            store_row<Q>(dst + 32 * q, wide, reinterpret_cast<const float *>(v), f);
        }
    }
    if (partial) {
        __stcg(partial + tid, m);
        __stcg(partial + kRowsCta + tid, l);
    } else if (live && p.lse) {
        p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    return true;
}

// Row r of a half's bfloat16 queries to halves in place, brought to [1, 2) by a power of two; returns what its scores have to be
// multiplied with.
template <int D>
__device__ __forceinline__ float halve_row(uint8_t *q, int r)
{
    uint4 x[D / 8];
    uint32_t mag = 0;
#pragma unroll
    for (int g = 0; g < D / 8; g++) {
        x[g] = *reinterpret_cast<const uint4 *>(q + chunk_at(r, g));
#pragma unroll
        for (int i = 0; i < 4; i++) asm("max.u16x2 %0, %0, %1;" : "+r"(mag) : "r"((&x[g].x)[i] & 0x7fff7fffu));
    }
    float down, up;
    query_scale(max(mag & 0xffffu, mag >> 16), down, up);
#pragma unroll
    for (int g = 0; g < D / 8; g++) *reinterpret_cast<uint4 *>(q + chunk_at(r, g)) = scaled_halves(x[g], down);
    return up;
}

// Meeting point of the eight softmax warps, bounded like every wait.
template <typename SM>
__device__ __forceinline__ bool softmax_sync(SM &sm, uint32_t &joins, int *err)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.join);
    return wait_warp(sm, &sm.join, joins++ & 1, err);
}

template <int D, typename Q, int KV>
__device__ void softmax_role(Smem<D, KV> &sm, const Args &args, uint32_t tmem, int W, int S)
{
    const AttnParams &p = args.p;
    const int tid = threadIdx.x, h = tid >> 7;
    int *count = reinterpret_cast<int *>(p.ws);
    SplitWs ws;
    ws.data = reinterpret_cast<float *>(p.ws + kAttnCounters * sizeof(int));
    uint32_t tiles = 0, units = 0, all_units = 0, all_tiles = 0, joins = 0;
    for (int k = 0; const Unit *at = unit_of(sm, k, p.c.err); k++) {
        const Unit &u = *at;
        float *partial = u.pieces > 1 ? ws.slot(u.slot, D) : nullptr;
        if (u.tb == u.ta) {   // no token of the row tile sees a key
            if (tid < u.rows) {
                const float z[32] = {};
                const size_t row = row_index(p, u, tid);
                for (int d = 0; d < D; d += 32) store_row<Q>(p.out + row * D + d, false, z, 0.f);
                if (p.lse) p.lse[row] = -INFINITY;
            }
        } else {
            float q_up = 1.f;
            const bool in_place = queries_in_place<Q, KV>(args);
            if (in_place) {   // this thread's row of queries, as halves
                if (!wait_warp(sm, &sm.q_raw, all_units & 1, p.c.err)) return;
                if (h < u.halves) q_up = halve_row<D>(sm.q[h], tid & 127);
                tc::fence_smem_to_async();
                __syncwarp();
                if ((tid & 31) == 0) mbar_arrive(&sm.q_full[all_units & 1]);
            }
            if (h < u.halves && !softmax_unit<D, Q, KV>(sm, p, u, tmem, W, S, in_place, q_up, partial, tiles, units, all_units, all_tiles)) return;
            all_units++;
            all_tiles += u.tb - u.ta;
            if (partial) {
                // the last of a unit's CTAs joins the pieces, in their order
                __threadfence();
                if (!softmax_sync(sm, joins, p.c.err)) return;
                if (tid == 0) {
                    const int done = atomicAdd(count + u.group, 1);
                    sm.last = done == u.pieces - 1;
                    if (sm.last) count[u.group] = 0;   // ready for the next call
                    __threadfence();
                }
                if (!softmax_sync(sm, joins, p.c.err)) return;
                if (sm.last && tid < u.rows) join_row<D, Q, KV>(p, u, ws.slot(u.first, D) + tid);
                if (!softmax_sync(sm, joins, p.c.err)) return;   // sm.last is read
            }
        }
        unit_done(sm, k);
    }
}

// New tokens of sequence b and its row, 0 tokens where its offsets or its row do not fit (`report`: says so).
__device__ __forceinline__ SeqInfo prefill_seq(const AttnParams &p, int b, int &c0, bool report)
{
    SeqInfo s;
    s.row = s.len = s.n = 0;
    s.ok = false;
    c0 = p.cu[b];
    const int c1 = p.cu[b + 1], row = p.rows[b];
    if (c0 < 0 || c1 < c0 || c1 > p.total || c1 - c0 > p.T || (b > 0 && p.cu[b - 1] > c0)) {
        if (report) atomicOr(p.c.err, KDA_DEVERR_SEQLEN);
    } else if (c1 > c0) {
        s = seq_info(p.c, row, c1 - c0, 0x7fffffff, report);
        if (!s.ok) s.n = 0;
    }
    return s;
}

// ---- warp 13: units in order of their number, handed to the other roles a few ahead
template <typename SM>
__device__ void unit_role(SM &sm, const AttnParams &p, int W, int S)
{
    const PagedCache &c = p.c;
    const int lane = threadIdx.x & 31;
    int *counter = reinterpret_cast<int *>(p.ws) + kMaxSplitCtas;   // next unit, CTAs that are done
    const int kept = min(p.B, kTable);
    long long all = sm.before[kept];   // (2^36 at most)
    for (int b0 = kept; b0 < p.B; b0 += 32) {   // sequences past the table
        int c0, t = 0;
        if (b0 + lane < p.B) t = (prefill_seq(p, b0 + lane, c0, blockIdx.x == 0).n * p.G + kRowsCta - 1) / kRowsCta;
        all += __reduce_add_sync(~0u, t);
    }
    // More row tiles than `total` tokens have: offsets that decrease let sequences share tokens.  Nothing is done then, so
    // that tiles and units are counted in 32 bits below.
    if (all > (long long)p.total * p.G / kRowsCta + p.B) {
        if (blockIdx.x == 0 && lane == 0) atomicOr(c.err, KDA_DEVERR_SEQLEN);
        all = 0;
    }
    // Fewer units than CTAs: they are split over the keys.  (Splitting those of a partly filled last round as well
    // costs more than it saves: 16384 tokens in a 2048 window, 512 units for 152 CTAs, 125 us against 122.)
    const long long n_units = all * c.Hkv;
    const int splits = n_units > 0 && n_units * 2 <= gridDim.x ? min(kMaxSplits, (int)(gridDim.x / n_units)) : 1;
    const long long total = n_units * splits;
    long long idx = blockIdx.x;
    for (int k = 0;; k++) {
        const int slot = k % kUnits;
        Unit u;
        u.idx = -1;
        if (idx < total) {
            const long long unit = idx / splits;
            const int y = (int)(idx - unit * splits), x = (int)(unit / c.Hkv);
            u.h = (int)(unit - (long long)x * c.Hkv);
            u.slot = (int)idx;         // (used where splits > 1: fewer than the CTAs then)
            u.first = u.slot - y;
            u.group = (int)unit;
            const int want = (int)all - 1 - x;   // the last row tiles first: the longest of a causal prompt
            int b = -1, tile = 0;
            if (want < sm.before[kept]) {
                int a = 0, e = kept;        // the last sequence with before[] <= want, 32 at a time
                while (e - a > 1) {
                    const int step = (e - a + 31) / 32, at = a + lane * step;
                    const unsigned m = __ballot_sync(~0u, at < e && sm.before[at] <= want);
                    a += (31 - __clz(m)) * step;
                    e = min(e, a + step);
                }
                b = a;
                tile = want - sm.before[a];
            } else {
                int at = sm.before[kept];
                for (int b0 = kept; b0 < p.B && b < 0; b0 += 32) {
                    int c0, t = 0;
                    if (b0 + lane < p.B) t = (prefill_seq(p, b0 + lane, c0, false).n * p.G + kRowsCta - 1) / kRowsCta;
                    int inc = t;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int v = __shfl_up_sync(~0u, inc, o);
                        if (lane >= o) inc += v;
                    }
                    const unsigned m = __ballot_sync(~0u, want < at + inc);
                    if (m) {
                        const int src = __ffs(m) - 1;
                        b = b0 + src;
                        tile = want - at - __shfl_sync(~0u, inc - t, src);
                    }
                    at += __shfl_sync(~0u, inc, 31);
                }
            }
            SeqInfo s;
            if (b < kept) s.row = sm.seq[b].x, s.len = sm.seq[b].y, s.n = sm.seq[b].z, u.c0 = sm.seq[b].w;
            else s = prefill_seq(p, b, u.c0, false);
            u.idx = (int)idx;
            u.row = s.row;
            u.n = s.n;
            u.len = s.len;
            u.r0 = tile * kRowsCta;
            u.t0 = u.r0 / p.G;
            u.g0 = u.r0 - u.t0 * p.G;
            u.rows = min(kRowsCta, u.n * p.G - u.r0);
            u.halves = u.rows > kHalf ? 2 : 1;
            u.p_first = u.len - u.n + u.t0;
            u.p_last = u.len - u.n + (u.r0 + u.rows - 1) / p.G;
            const KeyRange<kKeys> kr(u.p_first, u.p_last, u.len, W, S);
            // This split's share of the key tiles; splits past the last piece have none.  A tile takes 1.5 us, and one
            // CTA joins the pieces at about 3 us each, so their best number grows with the root of the tiles
            // (64 tokens behind 4096, 8 key heads: 59 us in 16 pieces, 35 in 4; behind 16384: 78 us in 19, 60 in 8;
            // behind 1000, 8 tiles: 26 us in 4, 21 in one).
            int share = max(1, kr.count);
            if (splits > 1) share = max(kMinShare, max((kr.count + splits - 1) / splits, (int)ceilf(sqrtf(2.f * kr.count))));
            u.pieces = max(1, (kr.count + share - 1) / share);
            u.ta = min(kr.count, y * share);
            u.tb = min(kr.count, u.ta + share);
            if (y >= u.pieces) {   // nothing to do: take another
                int nxt = 0;
                if (lane == 0) nxt = atomicAdd(counter, 1);
                idx = (long long)gridDim.x + __shfl_sync(~0u, nxt, 0);
                k--;
                continue;
            }
        }
        if (k >= kUnits && !wait_warp(sm, &sm.u_empty[slot], (k / kUnits - 1) & 1, c.err)) break;
        if (lane == 0) {
            sm.unit[slot] = u;
            mbar_arrive(&sm.u_full[slot]);
        }
        __syncwarp();
        if (u.idx < 0) break;
        int nxt = 0;
        if (lane == 0) nxt = atomicAdd(counter, 1);
        idx = (long long)gridDim.x + __shfl_sync(~0u, nxt, 0);
    }
    // every CTA has taken its last number: the last one to say so leaves the counters ready for the next call
    if (lane == 0 && atomicAdd(counter + 1, 1) == (int)gridDim.x - 1) counter[0] = counter[1] = 0;
}

template <int D, typename Q, int KV>
__global__ void __launch_bounds__(kThreads, 1) kda_attn_prefill_kernel(const __grid_constant__ Args args)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // the swizzle repeats every 1024 bytes of the shared address
    Smem<D, KV> &sm = *reinterpret_cast<Smem<D, KV> *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const AttnParams &p = args.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int W = p.window > 0 ? p.window : 0x7fffffff, S = p.window > 0 ? p.sinks : 0;
    if (tid == 0) {
        for (int i = 0; i < 2; i++) mbar_init(&sm.q_full[i], queries_in_place<Q, KV>(args) ? kSoftmax / 32 : kLoaders);   // by the unit's parity
        mbar_init(&sm.q_empty, 1);
        mbar_init(&sm.join, kSoftmax / 32);
        mbar_init(&sm.drain, 1);
        mbar_init(&sm.q_raw, 1);
        for (int i = 0; i < Smem<D, KV>::kRaw; i++) {
            mbar_init(&sm.raw_full[i], 33);   // lane 0 of warp 14, and its lanes or their copies
            mbar_init(&sm.raw_empty[i], kLoaders / 32);
        }
        for (int i = 0; i < (int)Smem<D, KV>::kSlots; i++) {
            mbar_init(&sm.full[i], kLoaders);
            mbar_init(&sm.empty[i], 1);
        }
        for (int h = 0; h < 2; h++) {
            mbar_init(&sm.s_full[h], 1);
            mbar_init(&sm.p_full[h], kHalf / 32);
            mbar_init(&sm.o_full[h], 1);
        }
        for (int i = 0; i < kUnits; i++) {
            mbar_init(&sm.u_full[i], 1);
            mbar_init(&sm.u_empty[i], KV == kKvE2M1 ? 14 : 13);   // the warps of the other roles
        }
        sm.stop = 0;
        fence_mbar_init();
    }
    grid_dependency_wait();
    // after the wait: a kernel that this one waits for may still need the SM's tensor memory
    if (warp == 12) tc::tmem_alloc(&sm.tmem, 512);

    // ---- row tiles before each sequence, for the first kTable of them
    {
        static_assert(kTable == kThreads, "one sequence a thread");
        const int kept = min(p.B, kTable);
        int tiles = 0;
        if (tid < kept) {
            int c0;
            const SeqInfo q = prefill_seq(p, tid, c0, blockIdx.x == 0);
            sm.seq[tid] = make_int4(q.row, q.len, q.n, c0);
            tiles = (q.n * p.G + kRowsCta - 1) / kRowsCta;
        }
        int inc = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) sm.warp_sum[warp] = inc;
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
        int off = inc - tiles;
        for (int i = 0; i < warp; i++) off += sm.warp_sum[i];
        if (tid <= kept) sm.before[tid] = off;
        if (tid == kThreads - 1 && kept == kTable) sm.before[kTable] = off + tiles;
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
    }
    const uint32_t tmem = sm.tmem;
    if (warp < 8) {
        regs_inc<kRegsSoftmax>();
        softmax_role<D, Q, KV>(sm, args, tmem, W, S);
        __syncwarp();
        regs_dec<kRegs>();   // back to what the common code was compiled for
    } else if (warp < 12) {
        regs_dec<kRegsLoad>();
        load_role<D, Q, KV>(sm, args, W, S);
        __syncwarp();
        regs_inc<kRegs>();
    } else {
        regs_dec<kRegsMma>();
        if (warp == 12) mma_role<D, std::conditional_t<KV != kKv16, Half, Q>>(sm, __reduce_max_sync(~0u, tmem), p.c.err);
        else if (warp == 13) unit_role(sm, p, W, S);
        else if (KV == kKvE2M1 && warp == 14) fetch_role<D, Q, KV>(sm, args, W, S);
        __syncwarp();
        regs_inc<kRegs>();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (sm.stop) {   // a wait gave up: let what was issued finish before the memory goes back
        if (warp == 12) {
            if (elect_one()) tc::commit(&sm.drain);
            mbar_wait_bounded(&sm.drain, 0, kLimitNs);
        }
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
    }
    if (warp == 12) tc::tmem_dealloc(tmem, 512);
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

cudaError_t encode(CUtensorMap *map, const void *base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3])
{
    const EncodeTiled fn = encoder();
    if (!fn) return cudaErrorSymbolNotFound;
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_pages(CUtensorMap *map, const void *base, const PagedCache &c)
{
    const cuuint64_t row = (cuuint64_t)c.D * 2;
    return encode(map, base, {(cuuint64_t)c.D, (cuuint64_t)c.Hkv * c.ps, (cuuint64_t)c.layers * c.pages}, {row, row * c.Hkv * c.ps},
                  {64, (cuuint32_t)c.ps, 1});
}

// Queries as [token][head][D].  A map wants strides under 2^40 bytes, not 0, each a multiple of the one before it; queries
// that have others (heads that share memory, heads farther apart than tokens), or that the encoder refuses for any
// other reason, take the copies (4 x 4096 tokens: 445 us against 406 when the map came in).  A dimension of one
// element may come with any stride, 0 too: it is not used.
bool map_queries(CUtensorMap *map, const AttnParams &p)
{
    if (kHalf % p.G) return false;
    const bool heads = p.Hq > 1, tokens = p.total > 1;
    const long long most = 1ll << 38, head = heads ? p.ql.head : 8, token = tokens ? p.ql.token : head * p.Hq;
    if (head <= 0 || head > most || token <= 0 || token > most || token % head) return false;
    return encode(map, p.q, {(cuuint64_t)p.c.D, (cuuint64_t)p.Hq, (cuuint64_t)p.total}, {(cuuint64_t)head * 2, (cuuint64_t)token * 2},
                  {64, (cuuint32_t)p.G, (cuuint32_t)(kHalf / p.G)}) == cudaSuccess;
}

template <int D, typename Q, int KV>
cudaError_t launch_as(const AttnParams &p, cudaStream_t stream)
{
    static KernelSetup setup;
    constexpr size_t smem = sizeof(Smem<D, KV>) + 1024;
    cudaError_t e = setup.get(kda_attn_prefill_kernel<D, Q, KV>, kThreads, smem, 0, nullptr);
    if (e != cudaSuccess) return e;
    int sms = 0;
    if ((e = paged_sm_count(&sms)) != cudaSuccess) return e;
    // row tiles of all sequences: at most one partly filled tile each
    const long long by_total = (long long)p.total * p.G / kRowsCta + p.B;
    const long long by_len = (long long)p.B * (((long long)p.T * p.G + kRowsCta - 1) / kRowsCta);
    const long long tiles = by_total < by_len ? by_total : by_len, units = tiles * p.c.Hkv;
    if (units > 0x7fffffffll) return cudaErrorInvalidValue;
    Args a = {};
    a.p = p;
    if (KV == kKv16 && ((e = encode_pages(&a.k, p.c.k, p.c)) != cudaSuccess || (e = encode_pages(&a.v, p.c.v, p.c)) != cudaSuccess)) return e;
    a.q_map = map_queries(&a.q, p);
    a.p.inv_g = 1.f / p.G;
    const int ctas = sms < kMaxSplitCtas ? sms : kMaxSplitCtas;
    return launch_pdl(kda_attn_prefill_kernel<D, Q, KV>, dim3((unsigned)ctas), dim3(kThreads), smem, stream, a);
}

template <int KV>
cudaError_t launch_kind(const AttnParams &p, cudaStream_t stream)
{
    if (p.c.D == 128) return p.f16 ? launch_as<128, Half, KV>(p, stream) : launch_as<128, Bf16, KV>(p, stream);
    return p.f16 ? launch_as<64, Half, KV>(p, stream) : launch_as<64, Bf16, KV>(p, stream);
}

}  // namespace

#ifdef KDA_PREFILL_E2M1   // a translation unit of its own (kda_attn_prefill_e2m1.cu), compiled beside the other's
cudaError_t launch_attn_prefill_e2m1(const AttnParams &p, cudaStream_t stream) { return launch_kind<kKvE2M1>(p, stream); }
#else
size_t attn_prefill_workspace(int D) { return kAttnCounters * sizeof(int) + kMaxSplitCtas * SplitWs::slot_floats(D) * sizeof(float); }

cudaError_t launch_attn_prefill(const AttnParams &p, cudaStream_t stream)
{
    return p.c.dtype == KDA_T_E2M1   ? launch_attn_prefill_e2m1(p, stream)
           : p.c.dtype == KDA_T_E4M3 ? launch_kind<kKvE4M3>(p, stream)
                                     : launch_kind<kKv16>(p, stream);
}
#endif

}  // namespace kda
