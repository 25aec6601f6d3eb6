"""The paged cache and its attention on the GPU against the 64-bit references of paged_ref.py.

Whatever no row holds is NaN in these caches (ends of pages, free pages), and table entries that no token
needs are -1 or out of range, so a kernel that reads past a row's end, or lets what it reads there into a
sum, shows it."""
from __future__ import annotations

import random

import pytest
import torch

from paged_ref import F64, PageModel, attention, check_attention, make_cache, spread

pytestmark = pytest.mark.gpu

BF, FH, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def queries(shape, dtype, seed):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * 1.3).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_decode(K, lens, T, Hkv, G, D, ps, dtype, kv, window=0, sinks=0, seed=0, n_tokens=None, layers=1, layer=0, scale=None):
    cache, dense = make_cache(K, lens, Hkv, D, ps, kv, seed, layers, layer)
    B = len(lens)
    order = list(range(B))
    random.Random(seed).shuffle(order)
    q = queries((B, T, Hkv * G, D), dtype, seed + 1)
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    lse = torch.full(q.shape[:-1], 7.0, device="cuda")
    nt = None if n_tokens is None else i32(n_tokens)
    K.kda_attn_decode(cache, layer, i32(order), q.cuda(), scale=scale, window=window, sinks=sinks, n_tokens=nt, out=out, lse=lse)
    assert K.kda_kv_get_error(cache) == 0
    for b, row in enumerate(order):
        n = T if n_tokens is None else n_tokens[b]
        ref = attention(q[b, :n].to(F64), *dense[row], lens[row], D ** -0.5 if scale is None else scale, window, sinks)
        check_attention(out[b, :n], lse[b, :n], ref, dtype, lens[row])
        assert (out[b, n:] == 7).all() and (lse[b, n:] == 7).all()   # entries past n_tokens stay
    return cache, q, out, lse


TYPES = [(BF, BF), (FH, FH), (BF, E4), (FH, E4)]
IDS = ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3"]


@pytest.mark.parametrize("dtype,kv", TYPES, ids=IDS)
@pytest.mark.parametrize("D,ps", [(128, 64), (64, 16), (128, 16), (64, 128)])
@pytest.mark.parametrize("T,Hkv,G", [(1, 2, 1), (1, 1, 5), (1, 2, 8), (3, 2, 5), (4, 1, 8), (16, 1, 3)])
def test_decode(K, dtype, kv, D, ps, T, Hkv, G):
    lens = [max(T, n) for n in spread(7, 700, D + ps + T)]
    run_decode(K, lens, T, Hkv, G, D, ps, dtype, kv, seed=T + G)


@pytest.mark.parametrize("dtype,kv", TYPES, ids=IDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 4), (17, 0), (100, 19), (64, 64), (5000, 7), (3, 5000)])
@pytest.mark.parametrize("T,G", [(1, 4), (5, 3)])
def test_decode_window(K, dtype, kv, window, sinks, T, G):
    lens = [max(T, n) for n in spread(6, 900, window + sinks + T)]
    run_decode(K, lens, T, 2, G, 128, 32, dtype, kv, window, sinks, seed=window)


@pytest.mark.parametrize("G,T", [(16, 1), (17, 1), (40, 1), (64, 1), (8, 16), (11, 7)])
def test_decode_many_rows(K, G, T):
    run_decode(K, [max(T, 130), max(T, 33)], T, 1, G, 64, 32, BF, BF, seed=G)


def test_decode_lengths_and_token_counts(K):
    """Rows without tokens, shorter than the call's tokens, and token counts from 0 to T."""
    for window, sinks in ((0, 0), (2, 1)):
        run_decode(K, [0, 1, 2, 3, 64, 0, 65], 4, 2, 3, 64, 16, BF, BF, window, sinks, seed=3)
        run_decode(K, [0, 1, 2, 3, 64, 90, 65], 4, 2, 3, 64, 16, FH, FH, window, sinks, seed=4, n_tokens=[0, 1, 2, 3, 4, 0, 2])


def test_decode_split_and_joined(K):
    """One long row over all CTAs (more pieces than are joined at once), next to short ones."""
    run_decode(K, [40000], 1, 1, 4, 128, 64, BF, BF, seed=1)
    run_decode(K, [30001, 1, 77], 2, 1, 3, 64, 16, FH, FH, seed=2)
    run_decode(K, [20011], 1, 1, 16, 128, 128, BF, E4, seed=3)


def test_decode_more_sequences_than_are_kept_on_chip(K):
    lens = [1 + (7 * i) % 40 for i in range(300)]
    run_decode(K, lens, 1, 1, 2, 64, 16, BF, BF, seed=5)


@pytest.mark.parametrize("T,G", [(1, 2), (4, 5), (16, 4)])
def test_decode_whole_units_and_cut_ones(K, T, G):
    """Runs of whole units (one or several a CTA, rows without tokens between them) and runs that cut them."""
    none = lambda B: [0 if i % 5 == 2 else T for i in range(B)]
    for lens in ([T + (11 * i) % 50 for i in range(90)], [T + 1000 - (i % 60) for i in range(40)], [T + 600] * 30 + [3000]):
        run_decode(K, lens, T, 8, G, 64, 16, FH, FH, seed=T, n_tokens=none(len(lens)))
    run_decode(K, [T + (7 * i) % 300 for i in range(280)], T, 2, G, 64, 16, BF, BF, 100, 3, seed=9, n_tokens=none(280))


def test_decode_layers_scale_and_extreme_scores(K):
    run_decode(K, [33, 100], 1, 2, 4, 64, 16, BF, BF, layers=3, layer=2, scale=0.0, seed=6)
    run_decode(K, [33, 100], 2, 2, 4, 128, 16, BF, BF, layers=3, layer=1, scale=3.0, seed=7)   # near one-hot rows
    run_decode(K, [65, 300], 1, 1, 4, 128, 64, BF, E4, scale=2.0, seed=8)


def test_decode_is_deterministic_and_replays_in_a_graph(K):
    cache, q, out, lse = run_decode(K, [5000, 17, 800, 1], 2, 2, 4, 128, 64, BF, BF, seed=9)
    order = list(range(4))
    random.Random(9).shuffle(order)
    rows, qd = i32(order), q.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, la = torch.empty_like(out), torch.empty_like(lse)
    with torch.cuda.stream(side):
        K.kda_attn_decode(cache, 0, rows, qd, out=a, lse=la)   # on another stream than its tensors' own
    side.synchronize()
    assert torch.equal(a, out) and torch.equal(la, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kda_attn_decode(cache, 0, rows, qd, out=a, lse=la)
    for _ in range(3):
        a.zero_()
        g.replay()
        assert torch.equal(a, out) and torch.equal(la, lse)


def test_decode_strided_queries_and_heads(K):
    cache, dense = make_cache(K, [50, 70, 9], 2, 64, 16, BF, 4)
    wide = queries((3, 2, 20, 64), BF, 5).cuda()
    rows = i32([0, 1, 2])
    for q in (wide[:, :, 4:12], wide[:, :, ::2][:, :, :8], wide.transpose(0, 1).contiguous().transpose(0, 1)[:, :, :4],
              wide[:, :1, 6:14]):
        out, lse = K.kda_attn_decode(cache, 0, rows, q, return_lse=True)
        for b in range(3):
            check_attention(out[b], lse[b], attention(q[b].cpu().to(F64), *dense[b], [50, 70, 9][b], 0.125, 0, 0), BF, 70)


def test_errors_leave_sequences_out(K):
    lens = [40, 50, 60, 70]
    cache, dense = make_cache(K, lens, 1, 64, 16, BF, 5)
    q = queries((4, 2, 2, 64), BF, 6).cuda()
    ref = K.kda_attn_decode(cache, 0, i32([0, 1, 2, 3]), q)
    # a row outside the table, a token count outside [0, T]
    for rows, n, bit in (([0, 99, 2, 3], None, 0x1), ([0, -1, 2, 3], None, 0x1), ([0, 1, 2, 3], [2, 3, 2, 2], 0x10),
                         ([0, 1, 2, 3], [2, -1, 2, 2], 0x10)):
        out = torch.full_like(ref, 5.0)
        K.kda_attn_decode(cache, 0, i32(rows), q, n_tokens=None if n is None else i32(n), out=out)
        assert K.kda_kv_get_error(cache) == bit
        assert (out[1] == 5).all() and all(torch.equal(out[i], ref[i]) for i in (0, 2, 3))
    # a length beyond the table
    keep = cache.seq_lens.clone()
    cache.seq_lens[1] = 1 << 20
    out = torch.full_like(ref, 5.0)
    K.kda_attn_decode(cache, 0, i32([0, 1, 2, 3]), q, out=out)
    assert K.kda_kv_get_error(cache) == 0x20
    assert (out[1] == 5).all() and all(torch.equal(out[i], ref[i]) for i in (0, 2, 3))
    cache.seq_lens.copy_(keep)
    # pages that the window has left behind may be gone, one that is needed may not
    cache.page_table[2, 0] = -1
    cache.page_table[3, 0] = 1 << 30
    out = K.kda_attn_decode(cache, 0, i32([0, 1, 2, 3]), q, window=20)
    assert K.kda_kv_get_error(cache) == 0
    for b in range(4):
        check_attention(out[b], None, attention(q[b].cpu().to(F64), *dense[b], lens[b], 0.125, 20, 0), BF, 70)
    K.kda_attn_decode(cache, 0, i32([0, 1, 2, 3]), q)
    assert K.kda_kv_get_error(cache) == 0x40
    assert K.kda_kv_get_error(cache) == 0


def run_prefill(K, new, total, Hkv, G, D, ps, dtype, kv, window=0, sinks=0, seed=0, scale=None):
    cache, dense = make_cache(K, total, Hkv, D, ps, kv, seed)
    B = len(new)
    order = list(range(B))
    random.Random(seed).shuffle(order)
    new_b = [new[r] for r in order]
    cu = [0]
    for n in new_b:
        cu.append(cu[-1] + n)
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


@pytest.mark.parametrize("dtype,kv", TYPES, ids=IDS)
@pytest.mark.parametrize("D,ps", [(128, 64), (64, 16), (128, 16), (64, 128), (128, 128), (128, 32)])
@pytest.mark.parametrize("Hkv,G", [(2, 1), (1, 5), (1, 8)])
def test_prefill(K, dtype, kv, D, ps, Hkv, G):
    new = [1, 130, 17, 0, 64]
    total = [1, 130, 150, 12, 333]
    run_prefill(K, new, total, Hkv, G, D, ps, dtype, kv, seed=D + ps + G)


@pytest.mark.parametrize("dtype,kv", TYPES, ids=IDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 4), (100, 19), (128, 128), (5000, 7), (3, 5000)])
def test_prefill_window(K, dtype, kv, window, sinks):
    run_prefill(K, [200, 33, 1, 90], [200, 500, 300, 700], 2, 3, 128, 32, dtype, kv, window, sinks, seed=window)


def test_prefill_tokens_before_the_row_begins(K):
    """More new tokens than the row holds: the first ones see nothing."""
    for window in (0, 5):
        run_prefill(K, [40, 300, 5], [20, 150, 0], 1, 2, 64, 16, BF, BF, window, 0, seed=11)
        run_prefill(K, [300], [0], 1, 2, 128, 16, FH, FH, window, 0, seed=12)


def test_prefill_longer(K):
    run_prefill(K, [700, 257], [1100, 257], 1, 4, 128, 64, BF, BF, seed=13)
    run_prefill(K, [600], [3000], 2, 1, 64, 16, FH, FH, seed=14)
    run_prefill(K, [64], [9000], 1, 4, 128, 64, BF, BF, seed=15)    # the key tiles split over CTAs
    run_prefill(K, [3], [5000], 1, 2, 64, 32, BF, E4, seed=16)
    run_prefill(K, [256], [300], 1, 64, 64, 32, BF, BF, seed=17)    # 64 heads a key head


def test_prefill_many_sequences(K):
    """More sequences than are kept on chip, and units enough for several a CTA."""
    n = [(5 * i) % 7 for i in range(600)]
    run_prefill(K, n, [x + (i % 30) for i, x in enumerate(n)], 1, 2, 64, 16, BF, BF, seed=18)
    n = [20 + i % 50 for i in range(40)]
    run_prefill(K, n, [x + (i % 90) for i, x in enumerate(n)], 8, 4, 64, 16, BF, BF, seed=19)


def test_prefill_scales(K):
    run_prefill(K, [100], [140], 1, 2, 128, 16, BF, BF, scale=0.0, seed=20)
    run_prefill(K, [100], [300], 1, 2, 128, 16, BF, BF, scale=3.0, seed=21)


def test_prefill_is_deterministic_and_replays_in_a_graph(K):
    cache, rows, cu, q, out, lse = run_prefill(K, [70, 40], [2000, 900], 1, 4, 128, 64, BF, BF, seed=22)
    a, la = torch.empty_like(out), torch.empty_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kda_attn_prefill(cache, 0, rows, cu, 70, q, out=a, lse=la)
    for _ in range(3):
        a.zero_()
        g.replay()
        assert torch.equal(a, out) and torch.equal(la, lse)
    # an output that is not on a 32-byte boundary
    buf = torch.empty(out.numel() + 8, dtype=out.dtype, device="cuda")[8:].view(out.shape)
    K.kda_attn_prefill(cache, 0, rows, cu, 70, q, out=buf)
    assert torch.equal(buf, out)


def test_prefill_errors_leave_sequences_out(K):
    cache, dense = make_cache(K, [60, 80, 50], 1, 64, 16, BF, 23)
    q = queries((90, 2, 64), BF, 24).cuda()
    rows = i32([0, 1, 2])
    ref = K.kda_attn_prefill(cache, 0, rows, i32([0, 30, 60, 90]), 30, q)
    assert K.kda_kv_get_error(cache) == 0
    for r, cu, most, bit, lost in (([0, 7, 2], [0, 30, 60, 90], 30, 0x1, [1]), ([0, 1, 2], [0, 30, 60, 90], 29, 0x20, [0, 1, 2]),
                                   ([0, 1, 2], [0, 30, 60, 91], 31, 0x20, [2]), ([0, 1, 2], [0, 60, 30, 90], 60, 0x20, None)):
        out = torch.full_like(ref, 5.0)
        K.kda_attn_prefill(cache, 0, i32(r), i32(cu), most, q, out=out)
        assert K.kda_kv_get_error(cache) == bit
        if lost is not None:
            for b in range(3):
                part = slice(30 * b, 30 * b + 30)
                assert (out[part] == 5).all() if b in lost else torch.equal(out[part], ref[part])


def test_prefill_equals_decode(K):
    """The same tokens by either call (the row blocks and orders of sums differ: to the outputs' rounding)."""
    cache, _ = make_cache(K, [100, 300], 2, 128, 32, BF, 25)
    q = queries((2, 8, 8, 128), BF, 26).cuda()
    a, la = K.kda_attn_decode(cache, 0, i32([0, 1]), q, window=90, sinks=3, return_lse=True)
    b, lb = K.kda_attn_prefill(cache, 0, i32([0, 1]), i32([0, 8, 16]), 8, q.flatten(0, 1), window=90, sinks=3, return_lse=True)
    assert (la.flatten(0, 1) - lb).abs().max() < 1e-5
    assert (a.flatten(0, 1).float() - b.float()).abs().max() <= 4 * 2.0 ** -8 * a.float().abs().max()


# ------------------------------------------------------------------------------------ pages

def same(K, cache, model):
    table = cache.page_table.cpu().tolist()
    for r, pages in enumerate(model.table):
        assert table[r] == pages + [-1] * (model.width - len(pages)), r
    assert cache.seq_lens.cpu().tolist() == model.lens
    assert cache.page_refs.cpu().tolist() == model.refs
    assert K.kda_kv_get_error(cache) == model.err
    model.err = 0


def contents(cache, model):
    """Every row's tokens carry the values that were written, in every layer, key and value."""
    k, v, table = cache.k.float().cpu(), cache.v.float().cpu(), cache.page_table.cpu()
    for layer in range(model.layers):
        for r, n in enumerate(model.lens):
            for pos in range(n):
                page = int(table[r, pos // model.ps])
                x = model.data[layer][page][pos % model.ps]
                if x is not None:
                    assert (k[layer, page, :, pos % model.ps] == x).all() and (v[layer, page, :, pos % model.ps] == -x).all()


@pytest.mark.parametrize("seed", range(6))
def test_page_calls_against_the_model(K, seed):
    r = random.Random(seed)
    ps, rows, width, pages, layers = r.choice([16, 32]), 12, 6, 40, 2
    cache = K.KdaKvCache.zeros(layers, pages, 2, rows, width, ps, 64, dtype=BF)
    model = PageModel(rows, width, pages, ps, layers)
    written = 0
    for step in range(40):
        op = r.choice(["extend", "extend", "append", "append", "truncate", "fork", "compact"])
        some = [r.randrange(rows) for _ in range(r.randint(1, 5))]
        if r.random() < 0.8:
            some = list(dict.fromkeys(some))   # else rows may be named twice
        if r.random() < 0.1:
            some[0] = r.choice([-1, rows, 1 << 30])
        if op == "extend":
            n = [r.choice([0, 1, 3, ps, 2 * ps + 1, -1 if r.random() < 0.1 else 2]) for _ in some]
            K.kda_kv_extend(cache, i32(some), i32(n))
            model.extend(some, n)
        elif op == "truncate":
            n = [r.randint(0, model.lens[x] if 0 <= x < rows else 5) + (r.random() < 0.1) for x in some]
            K.kda_kv_truncate(cache, i32(some), i32(n))
            model.truncate(some, n)
        elif op == "fork":
            src = [r.randrange(rows) for _ in some]
            K.kda_kv_fork(cache, i32(src), i32(some))
            model.fork(src, some)
        elif op == "compact":
            remap = K.kda_kv_compact(cache)
            assert remap.cpu().tolist() == model.compact()
        else:   # new tokens of rows that hold some, in fresh pages of their own, in both layers
            some = [x for x in dict.fromkeys(some) if 0 <= x < rows]
            K.kda_kv_extend(cache, i32(some), 2)
            before = list(model.lens)
            model.extend(some, [2] * len(some))
            some = [x for x in some if model.lens[x] == before[x] + 2]
            if some:
                vals = torch.arange(written, written + 2 * len(some)).view(-1, 2) % 200
                written += 2 * len(some)
                for layer in range(layers):
                    x = (vals + layer).to(BF)[:, :, None, None].expand(-1, -1, 2, 64).contiguous().cuda()
                    K.kda_kv_append(cache, layer, i32(some), x, -x)
                    for a, row in enumerate(some):
                        for t in range(2):
                            model.write(layer, row, model.lens[row] - 2 + t, float(vals[a, t] + layer))
        same(K, cache, model)
    contents(cache, model)


def test_extend_runs_out_of_pages(K):
    cache = K.KdaKvCache.zeros(1, 5, 1, 4, 8, 16, 64)
    model = PageModel(4, 8, 5, 16)
    for rows, n in (([0, 1], [40, 10]), ([2, 3], [33, 16]), ([2, 3, 0], [17, 0, 8]), ([3], [16]), ([0], [1000])):
        K.kda_kv_extend(cache, i32(rows), i32(n))
        model.extend(rows, n)
        same(K, cache, model)


def test_page_calls_at_scale(K):
    """Many pages and rows: scans and entries of several a thread."""
    rows, width, pages, ps = 3000, 40, 70001, 16
    cache = K.KdaKvCache.zeros(1, pages, 1, rows, width, ps, 64)
    model = PageModel(rows, width, pages, ps)
    r = random.Random(1)
    every = list(range(rows))
    n = [r.randint(0, 500) for _ in every]
    K.kda_kv_extend(cache, i32(every), i32(n))
    model.extend(every, n)
    same(K, cache, model)
    some = every[::2]
    cut = [r.randint(0, model.lens[x]) for x in some]
    K.kda_kv_truncate(cache, i32(some), i32(cut))
    model.truncate(some, cut)
    src, dst = every[1:1001:2], every[2:1002:2]
    K.kda_kv_fork(cache, i32(src), i32(dst))
    model.fork(src, dst)
    same(K, cache, model)
    K.kda_kv_extend(cache, i32(dst), 3)
    model.extend(dst, [3] * len(dst))
    same(K, cache, model)
    assert K.kda_kv_compact(cache).cpu().tolist() == model.compact()
    same(K, cache, model)


# ------------------------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype,kv", TYPES, ids=IDS)
@pytest.mark.parametrize("D,Hkv", [(64, 1), (128, 3), (128, 8), (64, 5)])
@pytest.mark.parametrize("form", ["even", "counts", "offsets"])
def test_append(K, dtype, kv, D, Hkv, form):
    new, old, ps = [3, 0, 1, 40, 17], [0, 5, 31, 20, 16], 16
    if form == "even":
        new = [3] * 5
    T, B = max(new), 5
    cache, _ = make_cache(K, [a + b for a, b in zip(old, new)], Hkv, D, ps, kv, 31, layers=2, layer=1)
    k0, v0 = cache.k.float().cpu(), cache.v.float().cpu()
    x = queries((B * T if form != "offsets" else sum(new), 2 * Hkv + 1, D), dtype, 32) * 3
    k, v = x[:, :Hkv].cuda(), x[:, Hkv + 1:].cuda()   # parts of one buffer
    big = x.cuda()
    k, v = big[:, :Hkv], big[:, Hkv + 1:]
    rows = [4, 0, 3, 1, 2]
    if form == "offsets":
        cu = [0]
        for r in rows:
            cu.append(cu[-1] + new[r])
        K.kda_kv_append(cache, 1, i32(rows), k, v, cu_seqlens=i32(cu))
        at = [[cu[b] + t for t in range(new[r])] for b, r in enumerate(rows)]
    elif form == "counts":
        K.kda_kv_append(cache, 1, i32(rows), k.unflatten(0, (B, T)), v.unflatten(0, (B, T)), n_tokens=i32([new[r] for r in rows]))
        at = [[b * T + t for t in range(new[r])] for b, r in enumerate(rows)]
    else:
        K.kda_kv_append(cache, 1, i32(rows), k, v)
        at = [[b * T + t for t in range(T)] for b in range(B)]
    assert K.kda_kv_get_error(cache) == 0
    table = cache.page_table.cpu()
    for name, before, sc, src in (("k", k0, cache.k_scale, k.cpu()), ("v", v0, cache.v_scale, v.cpu())):
        want = before.clone()
        for b, r in enumerate(rows):
            for t, i in enumerate(at[b]):
                pos = old[r] + t
                y = src[i].float()
                if kv == E4:
                    y = (y / sc[1].cpu()[:, None]).clamp(-448, 448).to(E4).float()
                want[1, int(table[r, pos // ps]), :, pos % ps] = y
        got = getattr(cache, name).float().cpu()
        assert torch.equal(got.nan_to_num(nan=1e30), want.nan_to_num(nan=1e30))


def test_append_special_values_and_scales(K):
    """Every half-precision value against several scales: codes as the IEEE quotient's, infinities clamped, NaN kept."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    for dtype in (BF, FH):
        x = every.view(dtype).view(64, 1, 16, 64).cuda()   # 64 rows, 16 heads
        scales = torch.tensor([1.0, 0.3, 1e-3, 7.1, 448.0, 3e-20, 1e20, 1.0000001, 0.9999999, 0.017, 2.0 ** -130, 3.0, 0.1, 65504.0, 1e-8, 5e-4])
        cache = K.KdaKvCache.zeros(1, 64, 16, 64, 1, 16, 64, dtype=E4, k_scale=scales.view(1, 16).cuda(), v_scale=scales.flip(0).view(1, 16).cuda())
        rows = torch.arange(64, dtype=torch.int32, device="cuda")
        K.kda_kv_extend(cache, rows, 1)
        K.kda_kv_append(cache, 0, rows, x, x)
        for got, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            got = got[0, :, :, 0].float()
            want = (x[:, 0].float() / s.view(1, 16, 1)).clamp(-448, 448).to(E4).float()
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.nan_to_num(nan=1e30), want.nan_to_num(nan=1e30))


def test_append_errors(K):
    cache, _ = make_cache(K, [20, 30, 3], 1, 64, 16, BF, 33)
    x = queries((3, 4, 1, 64), BF, 34).cuda()
    for change, bit in ((lambda c: c.seq_lens[2:3].fill_(3), 0x20), (lambda c: c.page_table[1, 1:2].fill_(-1), 0x40)):
        before = cache.k.clone()
        change(cache)
        K.kda_kv_append(cache, 0, i32([0, 1, 2]), x, x)
        assert K.kda_kv_get_error(cache) & bit
    K.kda_kv_append(cache, 0, i32([0, 50, 1]), x, x, n_tokens=i32([1, 1, 9]))
    assert K.kda_kv_get_error(cache) == 0x11


def test_offsets_past_32_bits(K):
    """Pages beyond 2^31 elements and 2^32 bytes of one tensor."""
    ps, Hkv, D = 128, 8, 128
    pages = (1 << 31) // (ps * Hkv * D) + 40
    kv = torch.empty(1, pages, Hkv, ps, D, dtype=BF, device="cuda")
    cache = K.KdaKvCache(k=kv, v=torch.empty_like(kv), page_table=torch.full((2, 4), -1, dtype=torch.int32, device="cuda"),
                         seq_lens=torch.zeros(2, dtype=torch.int32, device="cuda"), page_refs=torch.ones(pages, dtype=torch.int32, device="cuda"))
    cache.page_refs[-3:] = 0   # only the last pages are free
    K.kda_kv_extend(cache, i32([1]), 300)
    assert cache.page_table[1].tolist() == [pages - 3, pages - 2, pages - 1, -1]
    k, v = queries((300, Hkv, D), BF, 41), queries((300, Hkv, D), BF, 42)
    K.kda_kv_append(cache, 0, i32([1]), k.cuda(), v.cuda())
    q = queries((1, 1, 16, D), BF, 43)
    out, lse = K.kda_attn_decode(cache, 0, i32([1]), q.cuda(), return_lse=True)
    check_attention(out[0], lse[0], attention(q[0].to(F64), k.to(F64), v.to(F64), 300, D ** -0.5, 0, 0), BF, 300)
    qp = queries((300, 16, D), BF, 44)
    out, lse = K.kda_attn_prefill(cache, 0, i32([1]), i32([0, 300]), 300, qp.cuda(), return_lse=True)
    check_attention(out, lse, attention(qp.to(F64), k.to(F64), v.to(F64), 300, D ** -0.5, 0, 0), BF, 300)
    # a copy of the partly filled last page, and pages moved down from the end
    cache.page_refs[:4] = 0
    K.kda_kv_fork(cache, i32([1]), i32([0]))
    K.kda_kv_extend(cache, i32([0]), 1)
    assert cache.page_table[0].tolist() == [pages - 3, pages - 2, 0, -1] and K.kda_kv_get_error(cache) == 0
    assert torch.equal(cache.k[0, 0, :, :44], cache.k[0, pages - 1, :, :44])
    remap = K.kda_kv_compact(cache)
    assert remap[-3:].tolist() == [1, 2, 3]
    out2 = K.kda_attn_decode(cache, 0, i32([1]), q.cuda())
    assert torch.equal(out2, K.kda_attn_decode(cache, 0, i32([1]), q.cuda()))
    check_attention(out2[0], None, attention(q[0].to(F64), k.to(F64), v.to(F64), 300, D ** -0.5, 0, 0), BF, 300)


def test_a_cache_that_ends_with_its_tensor(K):
    """Whole caches of one page, one row, one token."""
    for ps in (16, 128):
        cache, dense = make_cache(K, [1], 1, 64, ps, BF, 51, extra_pages=0, extra_rows=0)
        q = queries((1, 1, 1, 64), BF, 52)
        out, lse = K.kda_attn_decode(cache, 0, i32([0]), q.cuda(), return_lse=True)
        check_attention(out[0], lse[0], attention(q[0].to(F64), *dense[0], 1, 0.125, 0, 0), BF, 1)
        out, lse = K.kda_attn_prefill(cache, 0, i32([0]), i32([0, 1]), 1, q[0].cuda(), return_lse=True)
        check_attention(out, lse, attention(q[0].to(F64), *dense[0], 1, 0.125, 0, 0), BF, 1)
