"""Rotary positions on the GPU against complex products in 64 bits (codes_ref.py)."""
from __future__ import annotations

import math
import random

import pytest
import torch

from codes_ref import GRID, make_cache4, nearest_code, token_codes, turn_error, turned
from paged_ref import EPS, F64, make_cache

pytestmark = pytest.mark.gpu

BF, FH, E4, U8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.uint8


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def freqs_of(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def data(shape, dtype, seed):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * 2).to(dtype)


def check(got, x, pos, freqs, interleaved, scale, dtype):
    """Half a step of the output's type, and FP32's errors before it (half's subnormals: steps of 2^-24)."""
    n = x.shape[:-2].numel()
    x, got = x.cpu().reshape(n, *x.shape[-2:]), got.cpu().reshape(n, *x.shape[-2:])
    ref = turned(x, pos.reshape(-1).cpu(), freqs, interleaved, scale)
    err = turn_error(x, 2 * len(freqs), interleaved, scale)
    tol = 1.001 * EPS[dtype] * (ref.abs() + err) + err + (2.0 ** -25 if dtype == FH else 0.0)
    off = (got.to(F64) - ref).abs()
    assert (off <= tol).all(), "off by up to %.3g of the tolerance" % (off / tol.clamp(min=1e-300)).max()
    rot = 2 * len(freqs)
    assert torch.equal(got[..., rot:], x[..., rot:])   # the rest of the head is the same bits


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "adjacent"])
@pytest.mark.parametrize("D,rot", [(16, 16), (64, 64), (64, 16), (64, 48), (80, 32), (128, 128), (128, 64), (128, 16), (96, 80), (256, 64), (512, 512)])
def test_rope(K, dtype, interleaved, D, rot):
    f = freqs_of(rot)
    rope = K.KdaRope.from_frequencies(f, interleaved, 1.25)
    for n, Hq, Hk in ((1, 1, 1), (7, 5, 2), (130, 12, 3)):
        q, k = data((n, Hq, D), dtype, n), data((n, Hk, D), dtype, n + 1)
        pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32)
        gq, gk = K.kda_rope(rope, pos.cuda(), q.cuda(), k.cuda())
        check(gq, q, pos, f, interleaved, 1.25, dtype)
        check(gk, k, pos, f, interleaved, 1.25, dtype)
        assert torch.equal(K.kda_rope(rope, pos.cuda(), q.cuda()), gq)


def test_positions_near_and_far(K):
    """0 gives the same bits, 2^31 - 1 and its negative the angle to 2^-24 of a turn; a negative position turns back."""
    f = freqs_of(64)
    rope = K.KdaRope.from_frequencies(f)
    pos = torch.tensor([0, 1, -1, 12345, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, -77], dtype=torch.int32)
    q = data((8, 3, 64), FH, 1)
    got = K.kda_rope(rope, pos.cuda(), q.cuda())
    assert torch.equal(got[0].cpu(), q[0])
    # 2^31 radians have 2^-22 of a radian in 64 bits of floating point: the reference's own error there
    err = 2.0 ** -22
    ref = turned(q, pos, f)
    tol = EPS[FH] * ref.abs() * 1.01 + turn_error(q, 64) + err * q.to(F64).abs().amax() * 2 + 2.0 ** -25
    assert ((got.cpu().to(F64) - ref).abs() <= tol).all()
    back = K.kda_rope(rope, (-pos[:4]).cuda(), got[:4])
    assert ((back.cpu().to(F64) - q[:4].to(F64)).abs() <= 4 * EPS[FH] * q[:4].to(F64).abs().amax()).all()
    # the angle of position 2^31 - 1 from exact integers
    from fractions import Fraction
    pi = Fraction(31415926535897932384626433832795028841971, 10 ** 40)
    x = torch.zeros(1, 1, 64, dtype=FH)
    x[0, 0, :32] = 1
    got = K.kda_rope(rope, i32([2 ** 31 - 1]), x.cuda()).cpu().to(F64)[0, 0]
    for i in range(32):
        turn = Fraction(f[i]) / (2 * pi) * (2 ** 31 - 1) % 1
        assert abs(float(got[i]) - math.cos(2 * math.pi * float(turn))) <= EPS[FH] + 2.0 ** -21
        assert abs(float(got[32 + i]) - math.sin(2 * math.pi * float(turn))) <= EPS[FH] + 2.0 ** -21


def test_empty_and_many(K):
    f = freqs_of(64)
    rope = K.KdaRope.from_frequencies(f)
    for shape in ((0, 4, 64), (3, 0, 4, 64), (0, 2, 4, 64)):
        q = torch.empty(shape, dtype=BF, device="cuda")
        assert K.kda_rope(rope, torch.empty(shape[:-2], dtype=torch.int32, device="cuda"), q).shape == shape
    q = data((5000, 3, 64), BF, 3)
    pos = torch.arange(5000, dtype=torch.int32)
    check(K.kda_rope(rope, pos.cuda(), q.cuda()), q, pos, f, False, 1.0, BF)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "adjacent"])
def test_layouts_and_in_place(K, interleaved):
    """[B, T, heads, D] in any strides, parts of one buffer, broadcast sources; outputs in place and in other strides; what lies
    between the heads of an output stays."""
    f = freqs_of(48)
    rope = K.KdaRope.from_frequencies(f, interleaved)
    wide = data((3, 5, 12, 64), BF, 5)
    pos = torch.randint(0, 9999, (3, 5), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    p = pos.cuda()
    for view in (lambda w: w[:, :, 2:9], lambda w: w[:, :, ::2], lambda w: w.transpose(0, 1).contiguous().transpose(0, 1)[:, :, :4],
                 lambda w: w[:, :, :1].expand(3, 5, 6, 64), lambda w: w.transpose(1, 2).contiguous().transpose(1, 2)):
        q = view(wide.cuda())
        got = K.kda_rope(rope, p, q)
        assert got.is_contiguous()
        check(got, view(wide), pos, f, interleaved, 1.0, BF)
    buf = wide.cuda()
    q, k = buf[:, :, :7], buf[:, :, 8:11]
    gq, gk = K.kda_rope(rope, p, q, k, q_out=q, k_out=k)
    assert gq is q and gk is k
    check(q, wide[:, :, :7], pos, f, interleaved, 1.0, BF)
    check(k, wide[:, :, 8:11], pos, f, interleaved, 1.0, BF)
    for h in (7, 11):
        assert torch.equal(buf[:, :, h].cpu(), wide[:, :, h])
    out = torch.full((5, 3, 14, 64), 3.0, dtype=BF, device="cuda")
    into = out.transpose(0, 1)[:, :, 1::2]
    K.kda_rope(rope, p, wide.cuda()[:, :, :7], q_out=into)
    check(into, wide[:, :, :7], pos, f, interleaved, 1.0, BF)
    assert (out[:, :, ::2] == 3).all()


def test_calls_of_like_forms(K):
    """Queries alone into a tensor that looks as keys would, then queries with such keys, and the other ways round."""
    f = freqs_of(64)
    rope = K.KdaRope.from_frequencies(f)
    x = data((4, 9, 3, 64), BF, 8)
    pos = torch.arange(9, dtype=torch.int32) * 77
    q, k, a, b = x.cuda()
    p = pos.cuda()
    for _ in range(2):
        assert K.kda_rope(rope, p, q, q_out=a) is a
        check(a, x[0], pos, f, False, 1.0, BF)
        gq, gk = K.kda_rope(rope, p, q, k)
        check(gq, x[0], pos, f, False, 1.0, BF)
        check(gk, x[1], pos, f, False, 1.0, BF)
        gq, gk = K.kda_rope(rope, p, q, k, k_out=b)
        assert gk is b and torch.equal(gq, a)
        gq, gk = K.kda_rope(rope, p, q, k, q_out=a)
        assert gq is a and torch.equal(gk, b)
        check(K.kda_rope(rope, p, q), x[0], pos, f, False, 1.0, BF)


def test_special_values(K):
    """A NaN or an infinity stays with its pair; the other pairs and the rest of the head are untouched by it."""
    f = freqs_of(32)
    rope = K.KdaRope.from_frequencies(f)
    q = data((2, 2, 64), BF, 6)
    q[0, 0, 3], q[0, 1, 40], q[1, 0, 20] = float("nan"), float("inf"), float("inf")
    got = K.kda_rope(rope, i32([9, 9]), q.cuda()).cpu()
    bad = torch.zeros(2, 2, 64, dtype=torch.bool)
    bad[0, 0, [3, 19]] = bad[1, 0, [4, 20]] = True
    assert torch.isnan(got[0, 0, [3, 19]]).all() and not torch.isfinite(got[1, 0, [4, 20]]).any()
    assert got[0, 1, 40] == float("inf")
    clean = torch.where(torch.isfinite(q), q, 0.0)
    ref = K.kda_rope(rope, i32([9, 9]), clean.cuda()).cpu()
    keep = ~bad
    keep[0, 1, 40] = False
    assert torch.equal(got[keep], ref[keep])


def test_streams_and_graphs(K):
    f = freqs_of(128)
    rope = K.KdaRope.from_frequencies(f)
    q, pos = data((33, 8, 128), BF, 7).cuda(), torch.arange(33, dtype=torch.int32, device="cuda") * 1000
    ref = K.kda_rope(rope, pos, q)
    side, out = torch.cuda.Stream(), torch.zeros_like(q)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        K.kda_rope(rope, pos, q, q_out=out)
    side.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kda_rope(rope, pos, q, q_out=out)
    for add in (0, 5):
        pos += add
        g.replay()
        assert torch.equal(out, K.kda_rope(rope, pos, q))


# ------------------------------------------------------------------------------------ append

def new_rows(form):
    new, old = ([3] * 5 if form == "even" else [3, 0, 1, 40, 17]), [0, 5, 31, 20, 16]
    return new, old, [4, 0, 3, 1, 2]


def append(K, cache, rope, form, q, k, v, new, rows, layer, q_out=None):
    """The call in one of its forms; returns what it returns, flat, and the places [row, t] of each new token in it."""
    T, B = max(new), 5
    if form == "offsets":
        cu = [0]
        for r in rows:
            cu.append(cu[-1] + new[r])
        got = K.kda_kv_append_rope(cache, layer, i32(rows), rope, q, k, v, cu_seqlens=i32(cu), q_out=q_out)
        return got, [(r, t, cu[b] + t) for b, r in enumerate(rows) for t in range(new[r])]
    if form == "counts":
        f = lambda x: None if x is None else x.unflatten(0, (B, T))
        got = K.kda_kv_append_rope(cache, layer, i32(rows), rope, f(q), f(k), f(v), n_tokens=i32([new[r] for r in rows]), q_out=f(q_out))
        return None if got is None else got.flatten(0, 1), [(r, t, b * T + t) for b, r in enumerate(rows) for t in range(new[r])]
    got = K.kda_kv_append_rope(cache, layer, i32(rows), rope, q, k, v, q_out=q_out)
    return got, [(r, t, b * T + t) for b, r in enumerate(rows) for t in range(T)]


KV = [(BF, BF), (FH, FH), (BF, E4), (FH, E4), (BF, U8), (FH, U8)]
KV_IDS = ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3", "bf16-e2m1", "fp16-e2m1"]


@pytest.mark.parametrize("dtype,kv", KV, ids=KV_IDS)
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (64, 16, False), (64, 48, False), (64, 32, True), (128, 128, False),
                                               (128, 128, True), (128, 80, False), (128, 32, False)])
@pytest.mark.parametrize("Hq,Hkv,form", [(4, 1, "even"), (15, 5, "counts"), (6, 3, "offsets")])
def test_append_rope(K, dtype, kv, D, rot, interleaved, Hq, Hkv, form):
    new, old, rows = new_rows(form)
    total, ps, layer = [a + b for a, b in zip(old, new)], 16, 1
    make = make_cache4 if kv == U8 else make_cache
    cache, _ = make(K, total, Hkv, D, ps, *(() if kv == U8 else (kv,)), 31, layers=2, layer=layer)
    before = cache.k.clone().view(U8), cache.v.clone().view(U8)
    f = freqs_of(rot)
    rope = K.KdaRope.from_frequencies(f, interleaved, 1.1)
    N = sum(new) if form == "offsets" else 5 * max(new)
    x = data((N, Hq + 2 * Hkv, D), dtype, 32)
    xd = x.cuda()
    q_out = torch.full((N, Hq, D), 7.0, dtype=dtype, device="cuda")
    _, at = append(K, cache, rope, form, xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], new, rows, layer, q_out=q_out)
    assert K.kda_kv_get_error(cache) == 0
    idx = torch.tensor([i for _, _, i in at])
    pos = torch.tensor([old[r] + t for r, t, _ in at], dtype=torch.int32)
    check(q_out[idx.cuda()], x[idx, :Hq], pos, f, interleaved, 1.1, dtype)
    rest = torch.ones(N, dtype=torch.bool)
    rest[idx] = False
    assert (q_out[rest.cuda()] == 7).all()   # tokens that do not count
    ref = turned(x[idx, Hq:Hq + Hkv], pos, f, interleaved, 1.1), x[idx, Hq + Hkv:].to(F64)
    err = turn_error(x[idx, Hq:Hq + Hkv], rot, interleaved, 1.1), torch.zeros(len(at), Hkv, D, dtype=F64)
    for which, (cached, scale) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        sc = torch.ones(Hkv, 1, dtype=F64) if scale is None else scale[layer].cpu().to(F64)[:, None]
        for i, (r, t, _) in enumerate(at):
            want, e = ref[which][i] / sc, err[which][i] / sc + (ref[which][i] / sc).abs() * 2.0 ** -24 * (kv in (E4, U8))
            if kv == U8:
                codes, s = (y[which] for y in token_codes(cache, layer, r, old[r] + t))
                block, eb = want.unflatten(-1, (-1, 16)), e.unflatten(-1, (-1, 16)).amax(-1)
                # the scale of a block is that of a largest magnitude within FP32's error of the exact one
                top, s = block.abs().amax(-1), s.to(F64)
                lo, hi = (((top + d * (eb + 2.0 ** -22 * top)) / 6).clamp(2.0 ** -9, 448.0).to(torch.float32).to(E4).to(F64) for d in (-1, 1))
                assert ((s >= lo) & (s <= hi)).all()
                # and each code a nearest one within that error
                y = block / s[..., None]
                near = (GRID - y.abs()[..., None]).abs().amin(-1)
                got = GRID[codes & 7] * (1 - 2 * (codes >> 3)).to(F64)
                over = (got.unflatten(-1, (-1, 16)) - y).abs() - near
                assert (over <= 2 * (eb / s)[..., None] + 2.0 ** -21 * y.abs() + 1e-12).all()
                if not (which == 0 and rot):
                    assert torch.equal(codes, torch.where(got == 0, codes, nearest_code((block / s[..., None]).flatten(-2).float())))
                continue
            page = int(cache.page_table[r, (old[r] + t) // ps])
            got = cached[layer, page, :, (old[r] + t) % ps].cpu().to(F64)
            if kv == E4:
                want = want.clamp(-448, 448)
                tol = 2.0 ** -4 * (want.abs() + e) + e + 2.0 ** -10   # half a step of codes, 2^-9 apart below 2^-6
            else:
                tol = 1.001 * EPS[kv] * (want.abs() + e) + e + (2.0 ** -25 if kv == FH else 0.0)
            assert ((got - want).abs() <= tol).all()
    # nothing else was written
    used = {(int(cache.page_table[r, (old[r] + t) // ps]), (old[r] + t) % ps) for r, t, _ in at}
    for was, now in zip(before, (cache.k.view(U8), cache.v.view(U8))):
        same = (was == now).flatten(3).cpu()     # [layers, pages, Hkv, bytes]
        assert same[0].all()
        touched = torch.zeros(same.shape[1], same.shape[3], dtype=torch.bool)
        for page, j in used:
            if kv == U8:
                touched[page, j * D // 2:(j + 1) * D // 2] = True
                touched[page, ps * D // 2 + j * D // 16:ps * D // 2 + (j + 1) * D // 16] = True
            else:
                w = same.shape[3] // ps
                touched[page, j * w:(j + 1) * w] = True
        assert (same[1] | touched[:, None]).all()


@pytest.mark.parametrize("kv", [BF, E4, U8], ids=["bf16", "e4m3", "e2m1"])
def test_append_rope_without_queries_and_in_place(K, kv):
    """Keys alone give the same cache; queries turned in place in their buffer; both equal the calls apart (16-bit cache)."""
    new, old, rows = new_rows("counts")
    total = [a + b for a, b in zip(old, new)]
    make = lambda: (make_cache4(K, total, 2, 64, 16, 41) if kv == U8 else make_cache(K, total, 2, 64, 16, kv, 41))[0]
    rope = K.KdaRope.make(64)
    x = data((200, 8, 64), BF, 42).cuda()
    a, b, c = make(), make(), make()
    got, at = append(K, a, rope, "counts", x[:, :4], x[:, 4:6], x[:, 6:], new, rows, 0)
    assert append(K, b, rope, "counts", None, x[:, 4:6], x[:, 6:], new, rows, 0)[0] is None
    buf = x.clone()
    append(K, c, rope, "counts", buf[:, :4], buf[:, 4:6], buf[:, 6:], new, rows, 0, q_out=buf[:, :4])
    idx = torch.tensor([i for _, _, i in at], device="cuda")
    assert torch.equal(buf[idx, :4], got[idx]) and torch.equal(buf[:, 4:], x[:, 4:])
    bits = lambda t: t.view(U8)
    for y in (b, c):
        assert torch.equal(bits(y.k), bits(a.k)) and torch.equal(bits(y.v), bits(a.v))
    pos = torch.zeros(200, dtype=torch.int32)
    for r, t, i in at:
        pos[i] = old[r] + t
    q, k = K.kda_rope(rope, pos.cuda(), x[:, :4], x[:, 4:6])
    assert torch.equal(q[idx], got[idx])
    if kv == BF:
        d = make()
        K.kda_kv_append(d, 0, i32(rows), k.unflatten(0, (5, 40)), x[:, 6:].unflatten(0, (5, 40)), n_tokens=i32([new[r] for r in rows]))
        assert torch.equal(bits(d.k), bits(a.k)) and torch.equal(bits(d.v), bits(a.v))


@pytest.mark.parametrize("kv", [BF, E4, U8], ids=["bf16", "e4m3", "e2m1"])
def test_append_rope_errors_leave_sequences_out(K, kv):
    lens = [40, 50, 60]
    make = lambda: (make_cache4(K, lens, 1, 64, 16, 51) if kv == U8 else make_cache(K, lens, 1, 64, 16, kv, 51))[0]
    rope = K.KdaRope.make(64)
    x = data((3, 2, 4, 64), BF, 52).cuda()
    good = make()
    ref = K.kda_kv_append_rope(good, 0, i32([0, 1, 2]), rope, x[:, :, :2], x[:, :, 2:3], x[:, :, 3:])
    assert K.kda_kv_get_error(good) == 0

    def damaged(what):
        cache = make()
        rows, n = [0, 1, 2], [2, 2, 2]
        if what == "row":
            rows[1] = 99
        elif what == "count":
            n[1] = 3
        elif what == "length":
            cache.seq_lens[1] = 1
        elif what == "page":
            cache.page_table[1, 3] = 1 << 30
        return cache, rows, n

    for what, bit in (("row", 0x1), ("count", 0x10), ("length", 0x20), ("page", 0x40)):
        cache, rows, n = damaged(what)
        out = torch.full_like(ref, 5.0)
        K.kda_kv_append_rope(cache, 0, i32(rows), rope, x[:, :, :2], x[:, :, 2:3], x[:, :, 3:], n_tokens=i32(n), q_out=out)
        assert K.kda_kv_get_error(cache) == bit
        assert (out[1] == 5).all() and torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
        pages = cache.page_table[1, :3].long()   # the row that was left out holds what it held
        assert torch.equal(cache.k.view(U8)[0, pages], make().k.view(U8)[0, pages])
        for r in (0, 2):
            p = cache.page_table[r, :-(-lens[r] // 16)].long()
            assert torch.equal(cache.k.view(U8)[0, p], good.k.view(U8)[0, p]) and torch.equal(cache.v.view(U8)[0, p], good.v.view(U8)[0, p])


def test_many_tokens_take_one_warp_each(K):
    """Enough tokens that a token's heads are not divided between warps."""
    n = 4000
    rope = K.KdaRope.make(128, scaling="yarn", factor=4.0)
    cache = K.KdaKvCache.zeros(1, n // 64 + 2, 2, 2, n // 64 + 2, 64, 128)
    K.kda_kv_extend(cache, i32([1]), n)
    x = data((1, n, 10, 128), BF, 61)
    xd = x.cuda()
    got = K.kda_kv_append_rope(cache, 0, i32([1]), rope, xd[:, :, :6], xd[:, :, 6:8], xd[:, :, 8:])
    assert K.kda_kv_get_error(cache) == 0
    f = [math.ldexp(float(t) % 2.0 ** 64, -64) * 2 * math.pi for t in rope.turns.tolist()]
    pos = torch.arange(n, dtype=torch.int32)
    check(got, x[:, :, :6], pos, f, False, rope.scale, BF)
    pages = cache.page_table[1, :-(-n // 64)].long()
    k = cache.k[0, pages].transpose(1, 2).flatten(0, 1)[:n]
    check(k, x[0, :, 6:8], pos, f, False, rope.scale, BF)
    assert torch.equal(cache.v[0, pages].transpose(1, 2).flatten(0, 1)[:n], xd[0, :, 8:])


def test_random_forms(K):
    """Calls of random forms on one cache, one after the other, against the calls apart."""
    r = random.Random(5)
    cache = K.KdaKvCache.zeros(1, 64, 2, 6, 10, 32, 64)
    twin = K.KdaKvCache.zeros(1, 64, 2, 6, 10, 32, 64)
    rope = K.KdaRope.make(32, interleaved=True)
    for step in range(25):
        rows = r.sample(range(6), r.randint(1, 6))
        T = r.choice([1, 2, 7])
        for c in (cache, twin):
            K.kda_kv_extend(c, i32(rows), T)
        x = data((len(rows), T, 7, 64), BF, 100 + step).cuda()
        a = K.kda_kv_append_rope(cache, 0, i32(rows), rope, x[:, :, :3], x[:, :, 3:5], x[:, :, 5:])
        pos = twin.seq_lens[i32(rows).long()][:, None] - T + torch.arange(T, device="cuda", dtype=torch.int32)
        q, k = K.kda_rope(rope, pos.int(), x[:, :, :3], x[:, :, 3:5])
        K.kda_kv_append(twin, 0, i32(rows), k, x[:, :, 5:])
        assert torch.equal(a, q)
        if int(cache.seq_lens.max()) > 300:
            for c in (cache, twin):
                K.kda_kv_truncate(c, i32(rows), i32([0] * len(rows)))
    assert torch.equal(cache.k, twin.k) and torch.equal(cache.v, twin.v)
    assert K.kda_kv_get_error(cache) == 0 and K.kda_kv_get_error(twin) == 0
