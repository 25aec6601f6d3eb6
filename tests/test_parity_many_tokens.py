"""Rotations and appends of so many tokens that a warp takes several passes over a token's heads, two in flight at once: the same
bits as calls so small that each pass has a warp of its own (those are held to the formulas in test_parity_rope.py and
test_parity_e2m1.py)."""
from __future__ import annotations

import pytest
import torch

from codes_ref import quantize, turned, turn_error, unpacked
from paged_ref import EPS, F64

pytestmark = pytest.mark.gpu

BF, FH, E4, U8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.uint8
PIECE = 61   # tokens of a small call: on any GPU of over 60 SMs every pass below has its own warp


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def data(shape, dtype, seed):
    return (torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)) * 2).to(dtype)


def bits(t):
    return t.view(torch.int16)


# heads, dims: passes of a token (32 lanes hold 512 elements of each of the two tensors)
FORMS = [(12, 8, 128, 128), (12, 3, 128, 48), (13, 5, 64, 64), (24, 9, 64, 16), (5, 2, 512, 512), (33, 40, 16, 16), (9, 4, 96, 96), (1, 1, 128, 128)]


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "adjacent"])
@pytest.mark.parametrize("Hq,Hk,D,rot", FORMS)
@pytest.mark.parametrize("n", [900, 3001])   # a few warps a token; one
def test_rope(K, dtype, interleaved, Hq, Hk, D, rot, n):
    freqs = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    rope = K.KdaRope.from_frequencies(freqs, interleaved, 1.25)
    x = data((n, Hq + Hk + 1, D), dtype, n + D)
    pos = torch.randint(-1000, 1 << 20, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32).cuda()
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk]
    gq, gk = K.kda_rope(rope, pos, q, k)
    for a in range(0, n, PIECE):
        sq, sk = K.kda_rope(rope, pos[a:a + PIECE], q[a:a + PIECE], k[a:a + PIECE])
        assert torch.equal(bits(gq[a:a + PIECE]), bits(sq)) and torch.equal(bits(gk[a:a + PIECE]), bits(sk)), a
    buf = x.clone()
    K.kda_rope(rope, pos, buf[:, :Hq], buf[:, Hq:Hq + Hk], q_out=buf[:, :Hq], k_out=buf[:, Hq:Hq + Hk])
    assert torch.equal(bits(buf[:, :Hq]), bits(gq)) and torch.equal(bits(buf[:, Hq:Hq + Hk]), bits(gk)) and torch.equal(bits(buf[:, -1]), bits(x[:, -1]))
    assert torch.equal(bits(K.kda_rope(rope, pos, q)), bits(gq))
    # and the formula, on every 50th token
    at = slice(0, None, 50)
    for got, src in ((gq, q), (gk, k)):
        got, src = got[at].cpu(), src[at].cpu()
        ref, err = turned(src, pos[at].cpu(), freqs, interleaved, 1.25), turn_error(src, rot, interleaved, 1.25)
        tol = 1.001 * EPS[dtype] * (ref.abs() + err) + err + (2.0 ** -25 if dtype == FH else 0.0)
        assert ((got.to(F64) - ref).abs() <= tol).all()


def held(cache, row, n):
    """What a row holds, by token: keys, then values (codes and block scales where there are 4 bits), as integers."""
    ps, D = cache.k.shape[3], cache.head_dim
    pages = cache.page_table[row, :-(-n // ps)].long()
    out = []
    for t in (cache.k, cache.v):
        x = t.view(U8)[1, pages]
        parts = (x,)
        if t.dtype == U8:
            codes, s = unpacked(x, D)
            parts = (codes, s.view(U8))
        out += [y.transpose(1, 2).flatten(0, 1)[:n] for y in parts]
    return out


def new_cache(K, kv, D, Hkv, ps, n, seed=3):
    width = -(-n // ps) + 1
    c = K.KdaKvCache.zeros(2, 3 * width, Hkv, 3, width, ps, D, dtype=kv)
    if c.k_scale is not None:   # another one for each head
        g = torch.Generator("cuda").manual_seed(seed)
        for s in (c.k_scale, c.v_scale):
            s.copy_((0.01 if kv == E4 else 0.3) * (1 + 3 * torch.rand(s.shape, device="cuda", generator=g)))
    return c


KV = [(BF, BF), (FH, FH), (BF, E4), (FH, E4), (BF, U8), (FH, U8)]
KV_IDS = ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3", "bf16-e2m1", "fp16-e2m1"]


@pytest.mark.parametrize("dtype,kv", KV, ids=KV_IDS)
@pytest.mark.parametrize("ps", [16, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,D,rot,interleaved", [(12, 8, 128, 128, False), (16, 5, 128, 80, False), (12, 8, 128, 64, True), (24, 9, 64, 64, False),
                                                      (9, 3, 64, 48, False), (40, 17, 64, 64, True)])
def test_append_rope(K, dtype, kv, ps, Hq, Hkv, D, rot, interleaved):
    lens, rows = [3000, 137], [2, 0]
    n = sum(lens)
    rope = K.KdaRope.make(rot, interleaved=interleaved, scaling="linear", factor=3.0)
    x = data((n, Hq + 2 * Hkv, D), dtype, D + ps)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    big, small, apart = (new_cache(K, kv, D, Hkv, ps, max(lens)) for _ in range(3))
    K.kda_kv_extend(big, i32(rows), i32(lens))
    got = K.kda_kv_append_rope(big, 1, i32(rows), rope, q, k, v, cu_seqlens=i32([0, lens[0], n]))
    assert K.kda_kv_get_error(big) == 0
    at = 0
    for row, m in zip(rows, lens):
        for a in range(at, at + m, PIECE):
            part = slice(a, min(a + PIECE, at + m))
            K.kda_kv_extend(small, i32([row]), part.stop - part.start)
            ref = K.kda_kv_append_rope(small, 1, i32([row]), rope, q[part], k[part], v[part])
            assert torch.equal(bits(got[part]), bits(ref)), a
        at += m
    for row, m in zip(rows, lens):
        for x0, x1 in zip(held(big, row, m), held(small, row, m)):
            assert torch.equal(x0, x1)
    for t in (big.k, big.v, small.k, small.v):
        assert not t.view(U8)[0].any()   # the other layer
    # keys alone, and queries in place
    buf = x.clone()
    K.kda_kv_extend(apart, i32(rows), i32(lens))
    K.kda_kv_append_rope(apart, 1, i32(rows), rope, None, k, v, cu_seqlens=i32([0, lens[0], n]))
    for row, m in zip(rows, lens):
        for x0, x1 in zip(held(big, row, m), held(apart, row, m)):
            assert torch.equal(x0, x1)
    K.kda_kv_append_rope(apart, 1, i32(rows), rope, buf[:, :Hq], buf[:, Hq:Hq + Hkv], buf[:, Hq + Hkv:], cu_seqlens=i32([0, lens[0], n]), q_out=buf[:, :Hq])
    assert torch.equal(bits(buf[:, :Hq]), bits(got)) and torch.equal(bits(buf[:, Hq:]), bits(x[:, Hq:]))
    for row, m in zip(rows, lens):
        for x0, x1 in zip(held(big, row, m), held(apart, row, m)):
            assert torch.equal(x0, x1)
    if kv == U8:   # values against the formula, on every page's first and last tokens
        at = 0
        for row, m in zip(rows, lens):
            pick = sorted({t for t in range(0, m) if t % ps in (0, ps - 1)})
            codes, s = (y.cpu()[pick] for y in held(big, row, m)[2:])
            want, ws = quantize(v[at:at + m].cpu()[pick].float(), big.v_scale[1].cpu()[:, None])
            assert torch.equal(s, ws.view(U8)) and torch.equal(codes, want)
            at += m


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
@pytest.mark.parametrize("ps,Hkv,D", [(16, 8, 128), (64, 5, 128), (128, 17, 64), (32, 3, 64)])
def test_append_to_4_bits(K, dtype, ps, Hkv, D):
    n = 3100
    x = data((n, 2 * Hkv, D), dtype, ps)
    big, small = (new_cache(K, U8, D, Hkv, ps, n) for _ in range(2))
    K.kda_kv_extend(big, i32([1]), n)
    K.kda_kv_append(big, 1, i32([1]), x[:, :Hkv], x[:, Hkv:])
    for a in range(0, n, PIECE):
        m = min(PIECE, n - a)
        K.kda_kv_extend(small, i32([1]), m)
        K.kda_kv_append(small, 1, i32([1]), x[a:a + m, :Hkv], x[a:a + m, Hkv:])
    both = held(big, 1, n), held(small, 1, n)
    for x0, x1 in zip(*both):
        assert torch.equal(x0, x1)
    for i, scale in enumerate((big.k_scale, big.v_scale)):
        want, ws = quantize(x[:, i * Hkv:(i + 1) * Hkv].cpu().float(), scale[1].cpu()[:, None])
        assert torch.equal(both[0][2 * i].cpu(), want) and torch.equal(both[0][2 * i + 1].cpu(), ws.view(U8))
    assert K.kda_kv_get_error(big) == 0 and K.kda_kv_get_error(small) == 0
