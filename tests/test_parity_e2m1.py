"""The 4-bit cache on the GPU: appended codes bit for bit, attention over them against the 64-bit formulas, page calls.

Whatever no row holds has NaN for its block scales, so a kernel that lets it reach a sum shows it."""
from __future__ import annotations

import random

import pytest
import torch

from codes_ref import GRID, make_cache4, nearest_code, quantize, token_codes, unpacked, values
from paged_ref import F64, attention, check_attention, spread

pytestmark = pytest.mark.gpu

BF, FH, E4, U8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.uint8


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def queries(shape, dtype, seed):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * 1.3).to(dtype)


# ------------------------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,Hkv,ps", [(64, 1, 16), (128, 3, 32), (128, 8, 128), (64, 5, 64)])
@pytest.mark.parametrize("form", ["even", "counts", "offsets"])
def test_append(K, dtype, D, Hkv, ps, form):
    """Codes and block scales are those of the documented FP32 steps, bit for bit; nothing else is written."""
    new, old = ([3] * 5 if form == "even" else [3, 0, 1, 40, 17]), [0, 5, 31, 20, 16]
    T, B, rows = max(new), 5, [4, 0, 3, 1, 2]
    cache, dense = make_cache4(K, [a + b for a, b in zip(old, new)], Hkv, D, ps, 31, layers=2, layer=1)
    was = cache.k.clone(), cache.v.clone()
    n = sum(new) if form == "offsets" else B * T
    x = (queries((n, 2 * Hkv + 1, D), dtype, 32).float() * torch.exp(2 * torch.randn(n, 2 * Hkv + 1, 1, generator=torch.Generator().manual_seed(33)))).to(dtype)
    big = x.cuda()
    k, v = big[:, :Hkv], big[:, Hkv + 1:]   # parts of one buffer
    if form == "offsets":
        cu = [0]
        for r in rows:
            cu.append(cu[-1] + new[r])
        K.kda_kv_append(cache, 1, i32(rows), k, v, cu_seqlens=i32(cu))
        at = [(r, t, cu[b] + t) for b, r in enumerate(rows) for t in range(new[r])]
    elif form == "counts":
        K.kda_kv_append(cache, 1, i32(rows), k.unflatten(0, (B, T)), v.unflatten(0, (B, T)), n_tokens=i32([new[r] for r in rows]))
        at = [(r, t, b * T + t) for b, r in enumerate(rows) for t in range(new[r])]
    else:
        K.kda_kv_append(cache, 1, i32(rows), k, v)
        at = [(r, t, b * T + t) for b, r in enumerate(rows) for t in range(T)]
    assert K.kda_kv_get_error(cache) == 0
    want = [c.cpu().clone() for c in was]
    for r, t, i in at:
        pos = old[r] + t
        page, j = int(cache.page_table[r, pos // ps]), pos % ps
        for w, y, sc in zip(want, (x[i, :Hkv], x[i, Hkv + 1:]), (cache.k_scale, cache.v_scale)):
            codes, s = quantize(y.float(), sc[1].cpu()[:, None])
            flat = w[1, page].flatten(1)
            flat[:, j * D // 2:(j + 1) * D // 2] = (codes[:, 0::2] | codes[:, 1::2] << 4).to(U8)
            flat[:, ps * D // 2 + j * D // 16:ps * D // 2 + (j + 1) * D // 16] = s.view(U8)
    assert torch.equal(cache.k.cpu(), want[0]) and torch.equal(cache.v.cpu(), want[1])


def test_append_special_values(K):
    """Zeros keep their sign, blocks of zeros and of tiny values the least scale; infinities and large values the largest one; a NaN
    takes its block, and no other; ties go to the even code."""
    cache = K.KdaKvCache.zeros(1, 2, 1, 1, 2, 16, 64, dtype=U8)
    K.kda_kv_extend(cache, i32([0]), 6)
    x = torch.zeros(6, 64)
    x[0, :4] = torch.tensor([0.0, -0.0, 1e-7, -1e-7])
    x[0, 16:20] = torch.tensor([6.0, 0.25, 0.75, -0.75])        # scale 1: ties 0.25 -> 0, 0.75 -> 1
    x[0, 32:38] = torch.tensor([6.0, 1.25, 1.75, 2.5, 3.5, 5.0])
    x[1, :3] = torch.tensor([float("inf"), 448.0 * 3, -448.0 * 6])
    x[1, 16] = -float("inf")
    x[2, 5] = float("nan")
    x[2, 16:32] = 1.0
    x[3] = 3e38                                                  # past the largest scale
    x[4, :16] = 2.0 ** -10                                       # a sixth of it is under the least scale
    x[5, :16] = torch.linspace(-5, 5, 16)
    x = x.to(BF)
    K.kda_kv_append(cache, 0, i32([0]), x.cuda()[:, None], x.cuda()[:, None])
    assert K.kda_kv_get_error(cache) == 0
    codes, s = unpacked(cache.k[0, int(cache.page_table[0, 0])].cpu(), 64)
    codes, s = codes[0, :6], s[0, :6].float()
    want_c, want_s = quantize(x.float(), torch.ones(1))
    nan = torch.isnan(want_s.float())
    assert torch.equal(torch.isnan(s), nan) and nan.sum() == 1 and nan[2, 0]
    assert torch.equal(s[~nan], want_s.float()[~nan])
    live = ~nan.repeat_interleave(16, -1)
    assert torch.equal(codes[live], want_c[live])
    assert codes[0, 1] == 8 and codes[0, 3] == 8 and s[0, 0] == 2.0 ** -9
    assert codes[0, 16:20].tolist() == [7, 0, 2, 10] and codes[0, 32:38].tolist() == [7, 2, 4, 4, 6, 6]
    assert s[1, 0] == 448 and codes[1, :3].tolist() == [7, 5, 15] and codes[1, 16] == 15
    assert (codes[3] == 7).all() and (s[3] == 448).all()
    assert (codes[4, :16] == 1).all()
    assert torch.equal(cache.v.cpu(), cache.k.cpu())


def test_append_scales_out_of_the_ordinary(K):
    """Layer scales whose reciprocals leave FP32's normal range, and 0."""
    for scale in (1e-30, 1e30, 0.0, 3.7e-5):
        cache = K.KdaKvCache.zeros(1, 1, 1, 1, 1, 16, 64, dtype=U8, k_scale=torch.full((1, 1), scale, device="cuda"),
                                   v_scale=torch.ones(1, 1, device="cuda"))
        K.kda_kv_extend(cache, i32([0]), 1)
        x = queries((1, 64), BF, 3)
        K.kda_kv_append(cache, 0, i32([0]), x.cuda()[:, None], x.cuda()[:, None])
        codes, s = unpacked(cache.k[0, 0].cpu(), 64)
        want_c, want_s = quantize(x.float(), torch.tensor([scale]))
        assert torch.equal(s[0, :1].float(), want_s.float()) and torch.equal(codes[0, :1], want_c)


# ------------------------------------------------------------------------------------ attention

def run_decode(K, lens, T, Hkv, G, D, ps, dtype, window=0, sinks=0, seed=0, n_tokens=None, layers=1, layer=0, scale=None):
    cache, dense = make_cache4(K, lens, Hkv, D, ps, seed, layers, layer)
    B = len(lens)
    order = list(range(B))
    random.Random(seed).shuffle(order)
    q = queries((B, T, Hkv * G, D), dtype, seed + 1)
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    lse = torch.full(q.shape[:-1], 7.0, device="cuda")
    K.kda_attn_decode(cache, layer, i32(order), q.cuda(), scale=scale, window=window, sinks=sinks,
                      n_tokens=None if n_tokens is None else i32(n_tokens), out=out, lse=lse)
    assert K.kda_kv_get_error(cache) == 0
    for b, row in enumerate(order):
        n = T if n_tokens is None else n_tokens[b]
        ref = attention(q[b, :n].to(F64), *dense[row], lens[row], D ** -0.5 if scale is None else scale, window, sinks)
        check_attention(out[b, :n], lse[b, :n], ref, dtype, lens[row])
        assert (out[b, n:] == 7).all() and (lse[b, n:] == 7).all()
    return cache, q, out, lse


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,ps", [(128, 64), (64, 16), (128, 16), (64, 128), (128, 32), (64, 32)])
@pytest.mark.parametrize("T,Hkv,G", [(1, 2, 1), (1, 1, 5), (1, 2, 8), (3, 2, 5), (4, 1, 5), (4, 1, 8), (16, 1, 3)])
def test_decode(K, dtype, D, ps, T, Hkv, G):
    lens = [max(T, n) for n in spread(7, 700, D + ps + T)]
    run_decode(K, lens, T, Hkv, G, D, ps, dtype, seed=T + G)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (FH, 64)], ids=["bf16", "fp16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 4), (17, 0), (100, 19), (64, 64), (5000, 7), (3, 5000)])
@pytest.mark.parametrize("T,G", [(1, 4), (5, 3)])
def test_decode_window(K, dtype, D, window, sinks, T, G):
    lens = [max(T, n) for n in spread(6, 900, window + sinks + T)]
    run_decode(K, lens, T, 2, G, D, 32, dtype, window, sinks, seed=window)


@pytest.mark.parametrize("G,T", [(16, 1), (17, 1), (40, 1), (64, 1), (8, 16), (11, 7)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_many_rows(K, G, T, D):
    run_decode(K, [max(T, 130), max(T, 33)], T, 1, G, D, 32, BF, seed=G)


def test_decode_lengths_and_token_counts(K):
    for window, sinks in ((0, 0), (2, 1)):
        run_decode(K, [0, 1, 2, 3, 64, 0, 65], 4, 2, 3, 64, 16, BF, window, sinks, seed=3)
        run_decode(K, [0, 1, 2, 3, 64, 90, 65], 4, 2, 3, 128, 16, FH, window, sinks, seed=4, n_tokens=[0, 1, 2, 3, 4, 0, 2])


def test_decode_split_and_joined(K):
    run_decode(K, [40000], 1, 1, 4, 128, 64, BF, seed=1)
    run_decode(K, [30001, 1, 77], 2, 1, 3, 64, 16, FH, seed=2)
    run_decode(K, [1 + (7 * i) % 40 for i in range(300)], 1, 1, 2, 64, 16, BF, seed=5)
    run_decode(K, [5 + (11 * i) % 50 for i in range(90)], 4, 8, 5, 64, 16, FH, seed=6)


def test_decode_layers_scale_and_extreme_scores(K):
    run_decode(K, [33, 100], 1, 2, 4, 64, 16, BF, layers=3, layer=2, scale=0.0, seed=6)
    run_decode(K, [33, 100], 2, 2, 4, 128, 16, BF, layers=3, layer=1, scale=3.0, seed=7)
    run_decode(K, [65, 300], 1, 1, 4, 128, 64, FH, scale=2.0, seed=8)


def test_decode_is_deterministic_and_replays_in_a_graph(K):
    cache, q, out, lse = run_decode(K, [5000, 17, 800, 1], 2, 2, 4, 128, 64, BF, seed=9)
    order = list(range(4))
    random.Random(9).shuffle(order)
    rows, qd = i32(order), q.cuda()
    a, la = torch.empty_like(out), torch.empty_like(lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        K.kda_attn_decode(cache, 0, rows, qd, out=a, lse=la)
    side.synchronize()
    assert torch.equal(a, out) and torch.equal(la, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kda_attn_decode(cache, 0, rows, qd, out=a, lse=la)
    for _ in range(3):
        a.zero_()
        g.replay()
        assert torch.equal(a, out) and torch.equal(la, lse)


def run_prefill(K, new, total, Hkv, G, D, ps, dtype, window=0, sinks=0, seed=0, scale=None):
    cache, dense = make_cache4(K, total, Hkv, D, ps, seed)
    B = len(new)
    order = list(range(B))
    random.Random(seed).shuffle(order)
    cu = [0]
    for r in order:
        cu.append(cu[-1] + new[r])
    wide = queries((cu[-1], Hkv * G + 2, D), dtype, seed + 1)
    q = wide[:, 1:-1]
    out, lse = K.kda_attn_prefill(cache, 0, i32(order), i32(cu), max(new), wide.cuda()[:, 1:-1], scale=scale, window=window, sinks=sinks,
                                  return_lse=True)
    assert K.kda_kv_get_error(cache) == 0
    for b, row in enumerate(order):
        part = slice(cu[b], cu[b + 1])
        ref = attention(q[part].to(F64), *dense[row], total[row], D ** -0.5 if scale is None else scale, window, sinks)
        check_attention(out[part], lse[part], ref, dtype, total[row])
    return cache, i32(order), i32(cu), wide.cuda()[:, 1:-1], out, lse


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,ps", [(128, 64), (64, 16), (128, 16), (64, 128), (128, 128), (128, 32), (64, 32)])
@pytest.mark.parametrize("Hkv,G", [(2, 1), (1, 5), (1, 8)])
def test_prefill(K, dtype, D, ps, Hkv, G):
    run_prefill(K, [1, 130, 17, 0, 64], [1, 130, 150, 12, 333], Hkv, G, D, ps, dtype, seed=D + ps + G)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (FH, 64)], ids=["bf16", "fp16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 4), (100, 19), (128, 128), (5000, 7), (3, 5000)])
def test_prefill_window(K, dtype, D, window, sinks):
    run_prefill(K, [200, 33, 1, 90], [200, 500, 300, 700], 2, 3, D, 32, dtype, window, sinks, seed=window)


def test_prefill_tokens_before_the_row_begins(K):
    for window in (0, 5):
        run_prefill(K, [40, 300, 5], [20, 150, 0], 1, 2, 64, 16, BF, window, 0, seed=11)
        run_prefill(K, [300], [0], 1, 2, 128, 16, FH, window, 0, seed=12)


def test_prefill_longer(K):
    run_prefill(K, [700, 257], [1100, 257], 1, 4, 128, 64, BF, seed=13)
    run_prefill(K, [600], [3000], 2, 1, 64, 16, FH, seed=14)
    run_prefill(K, [64], [9000], 1, 4, 128, 64, BF, seed=15)    # the key tiles split over CTAs
    run_prefill(K, [256], [300], 1, 64, 64, 32, BF, seed=17)
    n = [(5 * i) % 7 for i in range(600)]
    run_prefill(K, n, [x + (i % 30) for i, x in enumerate(n)], 1, 2, 64, 16, BF, seed=18)
    n = [20 + i % 50 for i in range(40)]
    run_prefill(K, n, [x + (i % 90) for i, x in enumerate(n)], 8, 4, 128, 16, BF, seed=19)


def test_prefill_is_deterministic_and_replays_in_a_graph(K):
    cache, rows, cu, q, out, lse = run_prefill(K, [70, 40], [2000, 900], 1, 4, 128, 64, BF, seed=22)
    a, la = torch.empty_like(out), torch.empty_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kda_attn_prefill(cache, 0, rows, cu, 70, q, out=a, lse=la)
    for _ in range(3):
        a.zero_()
        g.replay()
        assert torch.equal(a, out) and torch.equal(la, lse)


def test_missing_pages_are_left_out(K):
    """Keys that are seen but have no page count for nothing, with the error bit; pages that the window has left behind may be gone."""
    lens = [200, 300]
    cache, dense = make_cache4(K, lens, 1, 64, 16, 24)
    cache.page_table[0, 5] = -1
    cache.page_table[1, 0] = 1 << 30
    q = queries((2, 2, 3, 64), BF, 25)
    keep = [torch.ones(n, dtype=torch.bool) for n in lens]
    keep[0][80:96] = False
    keep[1][:16] = False
    flat = q.cuda().flatten(0, 1)
    for call in (lambda w: K.kda_attn_decode(cache, 0, i32([0, 1]), q.cuda(), window=w).flatten(0, 1),
                 lambda w: K.kda_attn_prefill(cache, 0, i32([0, 1]), i32([0, 2, 4]), 2, flat, window=w)):
        out = call(0)
        assert K.kda_kv_get_error(cache) == 0x40
        for b in range(2):
            k, v = (x[keep[b]] for x in dense[b])
            check_attention(out[2 * b:2 * b + 2], None, attention(q[b].to(F64), k, v, len(k), 0.125, 0, 0), BF, lens[b])
        out = call(90)
        assert K.kda_kv_get_error(cache) == 0
        for b in range(2):
            check_attention(out[2 * b:2 * b + 2], None, attention(q[b].to(F64), *dense[b], lens[b], 0.125, 90, 0), BF, lens[b])


def test_nan_shows(K):
    """A block with a NaN scale that a token sees makes its outputs NaN; a token that does not see it is not touched by decode of its row."""
    cache, dense = make_cache4(K, [100, 100], 1, 64, 16, 26)
    page = int(cache.page_table[0, 2])
    cache.k[0, page].view(-1)[16 * 32 + 4 * 4] = 0x7f   # token 36 of row 0, its first block
    q = queries((2, 1, 4, 64), BF, 27).cuda()
    out = K.kda_attn_decode(cache, 0, i32([0, 1]), q)
    assert torch.isnan(out[0]).all() and not torch.isnan(out[1]).any()
    out = K.kda_attn_decode(cache, 0, i32([0, 1]), q, window=60)
    assert not torch.isnan(out).any()
    out = K.kda_attn_prefill(cache, 0, i32([0, 1]), i32([0, 1, 2]), 1, q[:, 0])
    assert torch.isnan(out[0]).all() and not torch.isnan(out[1]).any()


# ------------------------------------------------------------------------------------ pages

def row_values(cache, layer, row):
    """A row's keys and values [len, Hkv, D] in 64 bits."""
    n, ps = int(cache.seq_lens[row]), cache.k.shape[3]
    got = []
    for x, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes, s = unpacked(x[layer, cache.page_table[row, :-(-n // ps)].long()].cpu(), cache.head_dim)
        y = values(codes, s, 1.0) * sc[layer].cpu().to(F64)[:, None, None]
        got.append(y.transpose(1, 2).flatten(0, 1)[:n])
    return got


@pytest.mark.parametrize("D,ps", [(64, 16), (128, 128), (128, 32)])
def test_pages_follow(K, D, ps):
    """Forks, copies of shared last pages, cuts and compaction keep every row's contents, in all layers."""
    r = random.Random(D + ps)
    cache = K.KdaKvCache.zeros(2, 64, 3, 8, 6, ps, D, dtype=U8)
    rows = list(range(8))
    held = {x: [[], []] for x in rows}   # row -> layers -> tokens

    def put(which, n, seed):
        K.kda_kv_extend(cache, i32(which), n)
        for layer in range(2):
            x = queries((len(which), n, 6, D), BF, seed + layer)
            K.kda_kv_append(cache, layer, i32(which), x.cuda()[:, :, :3], x.cuda()[:, :, 3:])
            for b, row in enumerate(which):
                for t in range(n):
                    both = [values(*quantize(y.float(), torch.ones(1)), 1.0) for y in (x[b, t, :3], x[b, t, 3:])]
                    held[row][layer] = held[row][layer] + [both]

    def check():
        assert K.kda_kv_get_error(cache) == 0
        for row in rows:
            assert int(cache.seq_lens[row]) == len(held[row][0])
            for layer in range(2):
                if held[row][layer]:
                    k, v = row_values(cache, layer, row)
                    assert torch.equal(k, torch.stack([t[0] for t in held[row][layer]])) and torch.equal(v, torch.stack([t[1] for t in held[row][layer]]))

    put([0, 1, 2], ps + 3, 1)
    check()
    K.kda_kv_fork(cache, i32([0, 0, 1]), i32([3, 4, 5]))
    for s, d in ((0, 3), (0, 4), (1, 5)):
        held[d] = [list(x) for x in held[s]]
    put([3, 4, 5, 0], 5, 10)     # into copies of the shared last pages
    check()
    cut = {0: 1, 3: ps + 2, 2: 0}
    K.kda_kv_truncate(cache, i32(list(cut)), i32(list(cut.values())))
    for row, n in cut.items():
        held[row] = [x[:n] for x in held[row]]
    K.kda_kv_compact(cache)
    check()
    put([0, 2, 4], r.randint(1, ps), 20)
    check()


def test_one_model_step_together(K):
    """Prompts rotated and appended, attended, forked, decoded and cut on one 4-bit cache: every attention call against the formulas on
    what the cache holds, and the whole captured step replayed."""
    D, Hq, Hkv, ps = 64, 6, 2, 16
    cache = K.KdaKvCache.zeros(1, 40, Hkv, 6, 8, ps, D, dtype=U8)
    cache.k_scale.fill_(0.5)
    rope = K.KdaRope.make(32, scaling="yarn", factor=2.0, original_len=64)
    x = queries((60, Hq + 2 * Hkv, D), BF, 70).cuda()
    cu, rows = i32([0, 23, 60]), i32([0, 1])
    K.kda_kv_extend(cache, rows, i32([23, 37]))
    q = K.kda_kv_append_rope(cache, 0, rows, rope, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cu_seqlens=cu)
    out, lse = K.kda_attn_prefill(cache, 0, rows, cu, 37, q, window=30, sinks=2, return_lse=True)
    for a, b, row in ((0, 23, 0), (23, 60, 1)):
        check_attention(out[a:b], lse[a:b], attention(q[a:b].cpu().to(F64), *row_values(cache, 0, row), b - a, D ** -0.5, 30, 2), BF, 60)
    K.kda_kv_fork(cache, i32([1, 1]), i32([2, 3]))
    rows = i32([0, 1, 2, 3])
    y = queries((4, 3, Hq + 2 * Hkv, D), BF, 71).cuda()
    one = torch.empty(4, 3, Hq, D, dtype=BF, device="cuda")
    turned = torch.empty_like(one)

    def step():
        K.kda_kv_extend(cache, rows, 3)
        K.kda_kv_append_rope(cache, 0, rows, rope, y[:, :, :Hq], y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:], q_out=turned)
        K.kda_attn_decode(cache, 0, rows, turned, out=one)

    def check():
        for b in range(4):
            n = int(cache.seq_lens[b])
            check_attention(one[b], None, attention(turned[b].cpu().to(F64), *row_values(cache, 0, b), n, D ** -0.5, 0, 0), BF, n)

    step()
    check()
    K.kda_kv_truncate(cache, rows, cache.seq_lens[rows.long()] - i32([0, 1, 2, 3]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        check()
    assert K.kda_kv_get_error(cache) == 0
