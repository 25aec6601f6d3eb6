// kda_rope.cu -- rotary positions: queries and keys turned by their positions (kda_rope), and on their way into the pages of
// a key-value cache (kda_kv_append_rope); also the append to a 4-bit cache.
//
// Mathematics.  Pair i of a head's first `rot` elements, (x_i, x_i + rot/2) or (x_2i, x_2i+1), is turned by the angle
// 2 pi position freq_i.  freq is held as a 64-bit fraction of a turn, so the product with the position modulo 2^64 is the
// exact fraction of a turn at any position: no table of angles, and no rounding that grows with the position (an
// angle of 2^20 radians in FP32 is off by 0.06).  Its top 32 bits as a float are off by 2^-25 of half a turn at most, the
// cosine and sine by 2^-23.
//
// Bound: HBM, every element is read and written once.  A warp takes a token; a lane takes the same two 16-byte
// pieces (eight pairs) of every 4th (head_dim 128) or 8th (64) head, so that it needs the same eight cosines and sines
// throughout.  They are worked out once by the warp (rot / 64 angles a lane) and shared through 4 rot bytes of shared
// memory a warp.  Calls of few tokens give each token several warps.
#include "kda_attn_common.cuh"
#include "kda_quant.cuh"

namespace kda {
namespace {

constexpr int kWarpsCta = 8;
// Heads of a lane whose pieces are on their way at once: two, in 24 warps an SM.  The rotation alone, each head followed by the next
// one's load: 4 x 4096 tokens 55.7 us (three 57.2, four in 16 warps 59).  The append, two at a time: 32000 tokens, queries kept,
// keys and values to E4M3 143 us (one in 32 warps 155, four in 16 warps 146), to 4 bits 171 us (176, 180).
constexpr int kAhead = 2;

template <typename Q>
__device__ __forceinline__ void unpack8(const uint4 &w, float *x)
{
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (Q::is_half) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = __uint_as_float(v[i] << 16), x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    }
}
template <typename Q>
__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(Q::pack(x[0], x[1]), Q::pack(x[2], x[3]), Q::pack(x[4], x[5]), Q::pack(x[6], x[7]));
}

// A lane's place in a head: its two pieces of 8 elements, and whether they are turned.
struct Place {
    int p0, p1;
    bool turned;
    __device__ Place(const Turns &r, int u)
    {
        const int R = r.rot >> 4;
        turned = u < R;
        p0 = turned && !r.adjacent ? u : 2 * u;
        p1 = turned && !r.adjacent ? u + R : 2 * u + 1;
    }
};

// Cosine and sine of angle f of a position to their places in the warp's shared memory (cosines, then sines).
__device__ __forceinline__ void angle(const Turns &r, int pos, unsigned long long freq, int f, float *cs)
{
    const long long turn = (long long)((unsigned long long)(long long)pos * freq);
    float s, c;
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
    cs[f] = c * r.scale;
    cs[r.rot / 2 + f] = s * r.scale;
}
// All angles of a position, by the warp.
__device__ __forceinline__ void angles(const Turns &r, int pos, float *cs, int lane)
{
    for (int f = lane; f < r.rot / 2; f += 32) angle(r, pos, __ldg(r.freq + f), f, cs);
    __syncwarp();
}

// A lane's eight cosines and sines.
struct Angles { float c[8], s[8]; };
__device__ __forceinline__ void load_angles(const Turns &r, const float *cs, int u, Angles &mine)
{
    const float4 *c = reinterpret_cast<const float4 *>(cs + 8 * u), *s = reinterpret_cast<const float4 *>(cs + r.rot / 2 + 8 * u);
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const float4 x = c[i], y = s[i];
        mine.c[4 * i] = x.x, mine.c[4 * i + 1] = x.y, mine.c[4 * i + 2] = x.z, mine.c[4 * i + 3] = x.w;
        mine.s[4 * i] = y.x, mine.s[4 * i + 1] = y.y, mine.s[4 * i + 2] = y.z, mine.s[4 * i + 3] = y.w;
    }
}

// Two pairs (a0, b0), (a1, b1) turned, two elements an instruction.
__device__ __forceinline__ void turn2(float &a0, float &a1, float &b0, float &b1, float c0, float c1, float s0, float s1)
{
    float t0, t1, u0, u1;
    tc::mul2(t0, t1, b0, b1, -s0, -s1);
    tc::mul2(u0, u1, a0, a1, s0, s1);
    tc::fma2(a0, a1, a0, a1, c0, c1, t0, t1);
    tc::fma2(b0, b1, b0, b1, c0, c1, u0, u1);
}
// Eight pairs turned: (x0[i], x1[i]), or the neighbours in x0 and then in x1.
__device__ __forceinline__ void turn8(float *x0, float *x1, const Angles &m, bool adjacent)
{
    if (adjacent) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            turn2(x0[2 * i], x0[2 * i + 2], x0[2 * i + 1], x0[2 * i + 3], m.c[i], m.c[i + 1], m.s[i], m.s[i + 1]);
            turn2(x1[2 * i], x1[2 * i + 2], x1[2 * i + 1], x1[2 * i + 3], m.c[4 + i], m.c[5 + i], m.s[4 + i], m.s[5 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) turn2(x0[i], x0[i + 1], x1[i], x1[i + 1], m.c[i], m.c[i + 1], m.s[i], m.s[i + 1]);
    }
}

template <typename Q>
__global__ void __launch_bounds__(kWarpsCta * 32, 3) kda_rope_kernel(const RopeParams p)
{
    extern __shared__ __align__(16) float all_angles[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long id = (long long)blockIdx.x * kWarpsCta + warp;
    const int part = (int)(id % p.parts);
    const long long tok = id / p.parts;
    grid_dependency_wait();
    if (tok >= p.tokens) return;
    float *cs = all_angles + warp * p.r.rot;
    const int log2 = p.lanes_log2, u = lane & ((1 << log2) - 1), per = 32 >> log2;   // heads of a pass
    const Place at(p.r, u);
    const bool used = u < p.D / 16;
    const int n0 = (p.x[0].heads + per - 1) / per, n = n0 + (p.x[1].heads + per - 1) / per;
    const long long seq = tok / p.T, in_seq = tok - seq * p.T;
    const int pos = __ldg(p.pos + tok);
    const uint16_t *src[kAhead];
    uint16_t *dst[kAhead];
    uint4 a[kAhead], b[kAhead];
    Angles mine;
    auto load = [&](int pass, int j) {
        dst[j] = nullptr;
        if (pass >= n || !used) return;
        const TurnedTensor &x = p.x[pass >= n0];
        const int h = (pass - (pass >= n0 ? n0 : 0)) * per + (lane >> log2);
        if (h >= x.heads) return;
        src[j] = x.src + seq * x.sl.seq + in_seq * x.sl.token + h * x.sl.head;
        dst[j] = x.dst + seq * x.dl.seq + in_seq * x.dl.token + h * x.dl.head;
        a[j] = __ldcs(reinterpret_cast<const uint4 *>(src[j]) + at.p0);
        b[j] = __ldcs(reinterpret_cast<const uint4 *>(src[j]) + at.p1);
    };
#pragma unroll
    for (int j = 0; j < kAhead; j++) load(part + j * p.parts, j);
    // while the first pieces are on their way
    angles(p.r, pos, cs, lane);
    if (at.turned) load_angles(p.r, cs, u, mine);
    for (int pass = part; pass < n; pass += kAhead * p.parts) {
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            if (dst[j]) {
                if (at.turned) {
                    float x0[8], x1[8];
                    unpack8<Q>(a[j], x0);
                    unpack8<Q>(b[j], x1);
                    turn8(x0, x1, mine, p.r.adjacent);
                    a[j] = pack8<Q>(x0);
                    b[j] = pack8<Q>(x1);
                }
                if (at.turned || src[j] != dst[j]) {   // (in place the rest stays)
                    __stcs(reinterpret_cast<uint4 *>(dst[j]) + at.p0, a[j]);
                    __stcs(reinterpret_cast<uint4 *>(dst[j]) + at.p1, b[j]);
                }
            }
            load(pass + (kAhead + j) * p.parts, j);   // its place is free again
        }
    }
}

// One piece of 8 elements (x, in FP32) into a head's row of a 16-bit or E4M3 cache.
template <typename Q, int KV>
__device__ __forceinline__ void put_piece(uint8_t *row, int piece, float *x, float2 scale)
{
    if constexpr (KV == kKv16) {
        reinterpret_cast<uint4 *>(row)[piece] = pack8<Q>(x);
    } else {
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = -x[i];
        neg_quotients8(x, scale, q);
        reinterpret_cast<uint2 *>(row)[piece] = e4m3x8(q);
    }
}

// A lane's two pieces (p0, p1) into a head of a 4-bit cache: `codes` and `scales` of the token.  A block is two
// neighbouring pieces; where a lane holds others (pairs half the rotated part apart), the partners' largest
// magnitudes come from the lanes that hold them.
__device__ __forceinline__ void put_blocks(uint8_t *codes, uint8_t *scales, const Place &at, int R, int lane, int lanes, float *x0, float *x1, float2 scale, bool used)
{
    float y0[8], y1[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x0[i] = -x0[i], x1[i] = -x1[i];
    neg_quotients8(x0, scale, y0);
    neg_quotients8(x1, scale, y1);
    const uint32_t m0 = magnitude8(y0), m1 = magnitude8(y1);
    const bool apart = at.p1 != at.p0 + 1;
    uint32_t b0 = max(m0, m1), b1 = b0;
    if (__any_sync(~0u, apart)) {
        // piece g < R is a lane's first, R <= g < 2 R a lane's second (2 R is even: partners stay below it)
        const int base = lane & ~(lanes - 1), g0 = at.p0 ^ 1, g1 = at.p1 ^ 1;
        const int l0 = base + (g0 < R ? g0 : g0 - R), l1 = base + (g1 < R ? g1 : g1 - R);
        const uint32_t a0 = __shfl_sync(~0u, m0, apart ? l0 : lane), a1 = __shfl_sync(~0u, m1, apart ? l0 : lane);
        const uint32_t c0 = __shfl_sync(~0u, m0, apart ? l1 : lane), c1 = __shfl_sync(~0u, m1, apart ? l1 : lane);
        if (apart) {
            b0 = max(m0, g0 < R ? a0 : a1);
            b1 = max(m1, g1 < R ? c0 : c1);
        }
    }
    if (!used) return;
    const uint32_t s0 = block_scale(b0), s1 = apart ? block_scale(b1) : s0;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; i++) y0[i] = -y0[i], y1[i] = -y1[i];
    neg_quotients8(y0, block_scale_value(s0), q);
    const uint32_t w0 = e2m1x8(q);
    neg_quotients8(y1, block_scale_value(s1), q);
    const uint32_t w1 = e2m1x8(q);
    if (apart) {
        reinterpret_cast<uint32_t *>(codes)[at.p0] = w0;
        reinterpret_cast<uint32_t *>(codes)[at.p1] = w1;
        if (!(at.p0 & 1)) scales[at.p0 >> 1] = (uint8_t)s0;
        if (!(at.p1 & 1)) scales[at.p1 >> 1] = (uint8_t)s1;
    } else {
        reinterpret_cast<uint2 *>(codes)[at.p0 >> 1] = make_uint2(w0, w1);
        scales[at.p0 >> 1] = (uint8_t)s0;
    }
}

// A warp for a token (or a part of its heads): queries turned into p.q.dst, keys turned into their page, values into theirs.
// 32000 tokens of 32 + 8 + 8 heads of 128 dims: 134 us to 16 bits, 143 to E4M3, 171 to 4 bits, 62 without rotation and queries
// (their bytes take 116, 107, 102, 25).  The chain of look-ups ahead of the data and the instructions bound it (issue slots 58 % busy, long
// scoreboard first among the stalls); at 80 registers every form also spills, 76 to 264 bytes of loads a thread.
template <typename Q, int KV, bool TURN>
__global__ void __launch_bounds__(kWarpsCta * 32, 3) kda_kv_append_turn_kernel(const AppendTurnParams p)
{
    __shared__ __align__(16) float all_angles[kWarpsCta][TURN ? 128 : 4];
    const AppendParams &ap = p.a;
    const PagedCache &c = ap.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long id = (long long)blockIdx.x * kWarpsCta + warp;
    const int part = (int)(id % p.parts);
    const long long tok = id / p.parts;
    const long long tokens = ap.cu ? ap.T : (long long)ap.B * ap.T;
    grid_dependency_wait();
    if (tok >= tokens) return;
    const int lanes = c.D / 16, u = lane & (lanes - 1), per = 32 / lanes, mine_h = lane / lanes;
    const Place at(p.r, u), plain = [&] { Place x = at; x.p0 = 2 * u; x.p1 = 2 * u + 1; x.turned = false; return x; }();
    const int nq = TURN ? (p.q.heads + per - 1) / per : 0, nk = (c.Hkv + per - 1) / per, n = nq + 2 * nk;
    const long long seq = ap.cu ? 0 : tok / ap.T, in_seq = tok - seq * ap.T;
    const long long row_k = (ap.cu ? 0 : seq * ap.kl.seq) + in_seq * ap.kl.token, row_v = (ap.cu ? 0 : seq * ap.vl.seq) + in_seq * ap.vl.token;
    const long long row_q = (ap.cu ? 0 : seq * p.q.sl.seq) + in_seq * p.q.sl.token, row_o = (ap.cu ? 0 : seq * p.q.dl.seq) + in_seq * p.q.dl.token;
    uint4 a[kAhead], b[kAhead];
    [[maybe_unused]] float layer_scale[kAhead];
    // pass: heads of the queries, then of the keys, then of the values
    auto head_of = [&](int pass) { return (pass < nq ? pass : pass < nq + nk ? pass - nq : pass - nq - nk) * per + mine_h; };
    auto load = [&](int pass, int j) {
        if (pass >= n) return;
        const int h = head_of(pass);
        if (h >= (pass < nq ? p.q.heads : c.Hkv)) return;
        const uint16_t *src = pass < nq ? p.q.src + row_q + h * p.q.sl.head : pass < nq + nk ? ap.k + row_k + h * ap.kl.head : ap.v + row_v + h * ap.vl.head;
        const Place &x = TURN && pass < nq + nk ? at : plain;
        if constexpr (KV != kKv16)
            if (pass >= nq) layer_scale[j] = __ldg((pass < nq + nk ? c.k_scale : c.v_scale) + ap.layer * c.Hkv + h);
        a[j] = __ldcs(reinterpret_cast<const uint4 *>(src) + x.p0);
        b[j] = __ldcs(reinterpret_cast<const uint4 *>(src) + x.p1);
    };
    // the first pieces, and the frequencies, are on their way while the token's place is found
#pragma unroll
    for (int j = 0; j < kAhead; j++) load(part + j * p.parts, j);
    unsigned long long freq[2] = {};   // (a cache's heads have 64 pairs at most)
    if constexpr (TURN) {
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (lane + 32 * i < p.r.rot / 2) freq[i] = __ldg(p.r.freq + lane + 32 * i);
    }
    int pos, page;
    if (!append_place(ap, tok, seq, in_seq, lane, lane == 0 && part == 0, pos, page)) return;
    [[maybe_unused]] Angles mine;
    if constexpr (TURN) {
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (lane + 32 * i < p.r.rot / 2) angle(p.r, pos, freq[i], lane + 32 * i, all_angles[warp]);
        __syncwarp();
        if (at.turned) load_angles(p.r, all_angles[warp], u, mine);
    }
    constexpr int SHIFT = KV == kKv16 ? 1 : 0;
    const int row_bytes = KV == kKvE2M1 ? c.D / 2 : c.D << SHIFT, in_page = pos & (c.ps - 1);
    const size_t head_bytes = (size_t)c.token_bytes() * c.ps;
    const size_t page_at = ((size_t)ap.layer * c.pages + page) * c.page_bytes();
    // a pass: `now` of the token's, in slot j
    auto put = [&](int now, int j) {
        const int h = head_of(now);
        const bool live = h < (now < nq ? p.q.heads : c.Hkv);
        const bool turned = TURN && now < nq + nk && at.turned;
        const Place &x = TURN && now < nq + nk ? at : plain;
        if (now < nq) {
            if (!live) return;
            uint16_t *dst = p.q.dst + row_o + h * p.q.dl.head;
            if (turned) {
                float x0[8], x1[8];
                unpack8<Q>(a[j], x0);
                unpack8<Q>(b[j], x1);
                turn8(x0, x1, mine, p.r.adjacent);
                a[j] = pack8<Q>(x0);
                b[j] = pack8<Q>(x1);
            }
            reinterpret_cast<uint4 *>(dst)[x.p0] = a[j];
            reinterpret_cast<uint4 *>(dst)[x.p1] = b[j];
            return;
        }
        const bool value = now >= nq + nk;
        uint8_t *head = (value ? c.v : c.k) + page_at + h * head_bytes;
        if constexpr (KV != kKvE2M1)
            if (!live) return;
        if (KV == kKv16 && !turned) {
            reinterpret_cast<uint4 *>(head + (size_t)in_page * row_bytes)[x.p0] = a[j];
            reinterpret_cast<uint4 *>(head + (size_t)in_page * row_bytes)[x.p1] = b[j];
            return;
        }
        float x0[8], x1[8];
        unpack8<Q>(a[j], x0);
        unpack8<Q>(b[j], x1);
        if (turned) turn8(x0, x1, mine, p.r.adjacent);
        float2 scale = make_float2(1.f, 1.f);
        if constexpr (KV != kKv16) scale = with_reciprocal(live ? layer_scale[j] : 1.f);
        if constexpr (KV == kKvE2M1) {
            put_blocks(head + (size_t)in_page * row_bytes, head + (size_t)c.ps * row_bytes + in_page * (c.D / 16), x, p.r.rot >> 4, lane, lanes, x0, x1, scale, live);
        } else {
            put_piece<Q, KV>(head + (size_t)in_page * row_bytes, x.p0, x0, scale);
            put_piece<Q, KV>(head + (size_t)in_page * row_bytes, x.p1, x1, scale);
        }
    };
    for (int pass = part; pass < n; pass += kAhead * p.parts) {
        if (pass != part) {
#pragma unroll
            for (int j = 0; j < kAhead; j++) load(pass + j * p.parts, j);
        }
#pragma unroll
        for (int j = 0; j < kAhead; j++)
            if (pass + j * p.parts < n) put(pass + j * p.parts, j);
    }
}

// Warps of a token: as many as its passes where there are few tokens (a pass each, the shortest chain), one where the
// tokens alone give every SM `kFill` warps.
constexpr int kFill = 16;
inline int parts_of(long long tokens, int passes, int sms)
{
    const long long want = ((long long)sms * kFill + tokens - 1) / tokens;
    return (int)(want < 1 ? 1 : want > passes ? passes : want);
}

template <typename Q, int KV, bool TURN>
cudaError_t append_as(const AppendTurnParams &p, long long warps, cudaStream_t stream)
{
    return launch_pdl(kda_kv_append_turn_kernel<Q, KV, TURN>, dim3((unsigned)((warps + kWarpsCta - 1) / kWarpsCta)), dim3(kWarpsCta * 32), 0, stream, p);
}
template <typename Q>
cudaError_t append_type(const AppendTurnParams &p, long long warps, cudaStream_t stream)
{
    if (!p.r.freq) return append_as<Q, kKvE2M1, false>(p, warps, stream);
    if (p.a.c.dtype == KDA_T_E2M1) return append_as<Q, kKvE2M1, true>(p, warps, stream);
    if (p.a.c.dtype == KDA_T_E4M3) return append_as<Q, kKvE4M3, true>(p, warps, stream);
    return append_as<Q, kKv16, true>(p, warps, stream);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, cudaStream_t stream)
{
    int sms = 0;
    const cudaError_t e = paged_sm_count(&sms);
    if (e != cudaSuccess) return e;
    p.lanes_log2 = 0;
    while (16 << p.lanes_log2 < p.D) p.lanes_log2++;
    const int per = 32 >> p.lanes_log2;
    p.parts = parts_of(p.tokens, (p.x[0].heads + per - 1) / per + (p.x[1].heads + per - 1) / per, sms);
    const long long warps = (long long)p.tokens * p.parts;
    const dim3 grid((unsigned)((warps + kWarpsCta - 1) / kWarpsCta));
    const size_t smem = (size_t)kWarpsCta * p.r.rot * sizeof(float);
    return p.f16 ? launch_pdl(kda_rope_kernel<Half>, grid, dim3(kWarpsCta * 32), smem, stream, p)
                 : launch_pdl(kda_rope_kernel<Bf16>, grid, dim3(kWarpsCta * 32), smem, stream, p);
}

cudaError_t launch_kv_append_turn(AppendTurnParams p, cudaStream_t stream)
{
    int sms = 0;
    const cudaError_t e = paged_sm_count(&sms);
    if (e != cudaSuccess) return e;
    const long long tokens = p.a.cu ? p.a.T : (long long)p.a.B * p.a.T;
    const int per = 512 / p.a.c.D;
    p.parts = parts_of(tokens, (p.q.heads + per - 1) / per + 2 * ((p.a.c.Hkv + per - 1) / per), sms);
    return p.a.f16 ? append_type<Half>(p, tokens * p.parts, stream) : append_type<Bf16>(p, tokens * p.parts, stream);
}

}  // namespace kda
