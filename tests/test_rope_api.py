"""Rotary positions and 4-bit caches without a GPU: the frequencies that KdaRope makes, and what the C entry points and their
binding refuse before anything is launched (no kernel ever sees the fake pointers)."""
from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import pytest
import torch

P = 0x10000   # a fake, aligned device pointer
TWO_PI = Fraction(62831853071795864769252867665590057683943, 10 ** 40)


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def msg(K):
    return K.library().kda_last_error().decode()


def ref(x):
    return None if x is None else ctypes.byref(x)


def layout(K, **kw):
    return K.paged._Layout(**{**dict(dtype=0, seq_stride=512, token_stride=128, head_stride=64), **kw})


def heads(K, n=2, src=None, dst=None):
    return K.rope._RopeLayout(n, src or layout(K), dst or layout(K))


def desc(K, **kw):
    return K.rope._RopeDesc(**{**dict(turns=P, rotary_dim=64, interleaved=0, scale=1.0), **kw})


def cache(K, **kw):
    d = dict(k=P, v=P, kv_dtype=0, num_layers=2, num_pages=8, num_kv_heads=2, page_size=16, head_dim=64, rows=4,
             max_pages=4, page_table=P, seq_lens=P, page_refs=P, k_scale=None, v_scale=None, err_word=P)
    return K.paged._Cache(**{**d, **kw})


def rope(K, d, D=64, pos=P, B=2, T=3, ql=None, q=P, qo=P, kl=None, k=P, ko=P):
    return K.library().kda_rope(ref(d), D, pos, B, T, ref(heads(K) if ql is None else ql), q, qo, ref(kl), k, ko, None)


def append(K, c, d, layer=0, rows=P, B=2, T=3, n=None, cu=None, ql=None, q=P, qo=P, k=P, kl=None, v=P, vl=None):
    kl, vl = layout(K) if kl is None else kl, layout(K) if vl is None else vl
    return K.library().kda_kv_append_rope(ref(c), layer, ref(d), rows, B, T, n, cu, ref(ql), q, qo, k, ref(kl), v, ref(vl), None)


BAD_ROPES = [(dict(rotary_dim=0), "rotary_dim", 2), (dict(rotary_dim=24), "rotary_dim", 2), (dict(rotary_dim=80), "rotary_dim", 2),
             (dict(rotary_dim=-16), "rotary_dim", 2), (dict(interleaved=2), "interleaved", 1), (dict(scale=float("nan")), "scale", 1),
             (dict(scale=float("inf")), "scale", 1), (dict(turns=None), "turns", 1), (dict(turns=P + 4), "turns", 1)]


@pytest.mark.parametrize("kw,word,status", BAD_ROPES, ids=lambda x: str(x)[:40])
def test_both_entries_check_the_rotation(K, kw, word, status):
    for call in (lambda: rope(K, desc(K, **kw)), lambda: append(K, cache(K), desc(K, **kw))):
        assert call() == status and word in msg(K)


BAD_HEADS = [(lambda K: heads(K, 0), "num_heads", 1), (lambda K: heads(K, 65537), "num_heads", 1),
             (lambda K: heads(K, src=layout(K, dtype=2)), "dtype", 1), (lambda K: heads(K, dst=layout(K, dtype=1)), "types", 1),
             (lambda K: heads(K, src=layout(K, token_stride=4)), "multiples of 8", 1), (lambda K: heads(K, dst=layout(K, head_stride=-64)), "negative", 1),
             (lambda K: heads(K, dst=layout(K, head_stride=0)), "share memory", 1), (lambda K: heads(K, dst=layout(K, token_stride=0)), "share memory", 1),
             (lambda K: heads(K, dst=layout(K, seq_stride=0)), "share memory", 1)]


@pytest.mark.parametrize("make,word,status", BAD_HEADS, ids=range(len(BAD_HEADS)))
def test_both_entries_check_the_heads(K, make, word, status):
    x = make(K)
    assert rope(K, desc(K), ql=x) == status and (word in msg(K) or "types" in msg(K))
    assert rope(K, desc(K), kl=x) == status
    c8 = cache(K, kv_dtype=2, k_scale=P, v_scale=P)
    assert append(K, c8, desc(K), ql=x) == status and (word in msg(K) or "types" in msg(K))


def test_rope_refusals(K):
    d = desc(K)
    for D in (0, 8, 72, 528):
        assert rope(K, d, D=D) == 2 and "head_dim" in msg(K)
    assert rope(K, None) == 1 and "rope is null" in msg(K)
    assert rope(K, d, B=-1) == 1 and rope(K, d, T=-1) == 1
    assert rope(K, d, B=1 << 20, T=1 << 12) == 2 and "31 bits" in msg(K)
    assert K.library().kda_rope(ref(d), 64, P, 1, 1, None, P, P, None, None, None, None) == 1 and "layout of q" in msg(K)
    for kw in (dict(pos=None), dict(pos=P + 2), dict(q=None), dict(q=P + 8), dict(qo=P + 4), dict(kl=heads(K), k=None), dict(kl=heads(K), ko=P + 8)):
        assert rope(K, d, **kw) == 1 and "aligned" in msg(K)
    assert rope(K, d, ql=heads(K, src=layout(K, dtype=1), dst=layout(K, dtype=1)), kl=heads(K)) == 1 and "different types" in msg(K)
    assert rope(K, d, B=0, pos=None, q=None) == 0 and rope(K, d, T=0, q=None) == 0


def test_append_rope_refusals(K):
    c, d = cache(K), desc(K)
    assert append(K, None, d) == 1 and append(K, c, None) == 1 and "rope is null" in msg(K)
    assert append(K, c, d, layer=2) == 1 and "layer" in msg(K)
    assert append(K, c, d, n=P, cu=P) == 1 and "exclude" in msg(K)
    assert append(K, c, d, B=1 << 20, T=1 << 12) == 2
    assert append(K, c, d, kl=layout(K, dtype=1), vl=layout(K, dtype=1)) == 1 and "cache holds" in msg(K)
    h16 = heads(K, src=layout(K, dtype=1), dst=layout(K, dtype=1))
    assert append(K, cache(K, kv_dtype=4, k_scale=P, v_scale=P), d, ql=h16) == 1 and "different types" in msg(K)
    for kw in (dict(rows=None), dict(k=P + 8), dict(v=None), dict(n=P + 1), dict(cu=P + 2), dict(ql=heads(K), q=None), dict(ql=heads(K), qo=P + 8)):
        assert append(K, c, d, **kw) == 1 and "aligned" in msg(K)
    # packed queries need no stride between sequences
    assert append(K, c, d, cu=P, ql=heads(K, dst=layout(K, seq_stride=0)), q=None) == 1 and "aligned" in msg(K)
    assert append(K, c, d, B=0) == 0 and append(K, c, d, T=0) == 0


def test_a_4_bit_cache_needs_its_scales(K):
    lib = K.library()
    for kw, word in ((dict(), "k_scale"), (dict(k_scale=P), "v_scale"), (dict(k_scale=P, v_scale=P + 2), "v_scale")):
        c = cache(K, kv_dtype=4, **kw)
        assert lib.kda_kv_append(ref(c), 0, P, 1, 1, None, None, P, ref(layout(K)), P, ref(layout(K)), None) == 1 and word in msg(K)
        assert append(K, c, desc(K)) == 1 and word in msg(K)
    c = cache(K, kv_dtype=4, k_scale=P, v_scale=P)
    assert lib.kda_kv_append(ref(c), 0, P, 1, 0, None, None, P, ref(layout(K)), P, ref(layout(K)), None) == 0
    assert lib.kda_attn_workspace_size(ref(c)) == lib.kda_attn_workspace_size(ref(cache(K)))


def test_binding_of_4_bit_caches(K):
    c = K.KdaKvCache.zeros(2, 4, 3, 2, 2, 16, 128, dtype=torch.uint8, device="cpu")
    assert c.k.shape == (2, 4, 3, 16, 72) and c.head_dim == 128 and c.Hkv == 3
    st = c.c_struct()
    assert (st.kv_dtype, st.head_dim, st.page_size) == (4, 128, 16) and st.k_scale and st.v_scale
    assert K.KdaKvCache.zeros(1, 4, 3, 2, 2, 16, 64, dtype=torch.uint8, device="cpu").k.shape[-1] == 36
    c.k_scale = None
    with pytest.raises(ValueError, match="4-bit"):
        c.c_struct()
    i32 = torch.int32
    for last in (64, 37):
        with pytest.raises(ValueError, match="4-bit"):
            K.KdaKvCache(torch.zeros(1, 2, 2, 16, last, dtype=torch.uint8), torch.zeros(1, 2, 2, 16, last, dtype=torch.uint8),
                         torch.zeros(1, 2, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(2, dtype=i32)).c_struct()


def test_binding_refusals(K):
    BF, i32 = torch.bfloat16, torch.int32
    r = K.KdaRope.make(32, device="cpu")
    q, k, pos = torch.zeros(3, 4, 64, dtype=BF), torch.zeros(3, 2, 64, dtype=BF), torch.zeros(3, dtype=i32)
    for bad in (dict(positions=pos.long()), dict(q=q.float()), dict(q=[0]), dict(k=[0]), dict(q_out=[0]), dict(k_out=[0])):
        with pytest.raises(TypeError):
            K.kda_rope(r, **{**dict(positions=pos, q=q, k=k), **bad})
    for bad in (dict(positions=pos[:2]), dict(positions=pos[None]), dict(q=q[None, None]), dict(q=q[0]), dict(k=k[:2]), dict(k=k.half()),
                dict(k=k[..., :32]), dict(q_out=q[:, :2]), dict(q_out=q.half()), dict(q=torch.zeros(3, 64, 4, dtype=BF).transpose(1, 2)),
                dict(k=None, k_out=k), dict(q=q.to("meta"), positions=pos)):
        with pytest.raises(ValueError):
            K.kda_rope(r, **{**dict(positions=pos, q=q, k=k), **bad})
    with pytest.raises(ValueError):
        K.kda_rope(K.KdaRope.make(32, device="meta"), pos, q)
    c = K.KdaKvCache.zeros(1, 4, 2, 3, 2, 16, 64, device="cpu")
    rows = torch.zeros(3, dtype=i32)
    for bad in (dict(q=q[:2]), dict(q=q.half()), dict(v=k[:2]), dict(q=q, k=k[:2], v=k[:2]), dict(q=None, q_out=q), dict(q_out=q[:, :1]),
                dict(rows=rows[:2]), dict(rows=[0]), dict(cu_seqlens=rows), dict(layer=1 << 40), dict(k=k[..., :32], v=k[..., :32])):
        with pytest.raises(ValueError):
            K.kda_kv_append_rope(**{**dict(cache=c, layer=0, rows=rows, rope=r, q=q, k=k, v=k), **bad})
    for bad in (dict(q=[0]), dict(k=0), dict(n_tokens=torch.zeros(3))):
        with pytest.raises(TypeError):
            K.kda_kv_append_rope(**{**dict(cache=c, layer=0, rows=rows, rope=r, q=q, k=k, v=k), **bad})
    with pytest.raises(ValueError, match="cu_seqlens"):
        K.kda_kv_append_rope(c, 0, rows[:1], r, None, k[None], k[None], cu_seqlens=rows[:2])


def test_frequencies_are_fractions_of_a_turn(K):
    """To 2^-64 of a turn, for frequencies of any size (whole turns drop out)."""
    f = [1.0, 0.5, 1e-4, 123.456, 1e9, -0.25, 0.0, 2.0 ** -70]
    r = K.KdaRope.from_frequencies(f, device="cpu")
    assert r.rotary_dim == 16 and r.turns.dtype == torch.int64
    for x, t in zip(f, r.turns.tolist()):
        want = Fraction(x) / TWO_PI * 2 ** 64
        off = (want - t) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(abs(x)) * Fraction(2 ** 64, 10 ** 40)
    assert torch.equal(K.KdaRope.from_frequencies(torch.tensor(f, dtype=torch.float64), device="cpu").turns, r.turns)
    for bad in (float("nan"), float("inf")):
        with pytest.raises(ValueError):
            K.KdaRope.from_frequencies([bad], device="cpu")


def radians(r):
    return [float(Fraction(t % 2 ** 64, 2 ** 64) * TWO_PI) for t in r.turns.tolist()]


def test_scalings(K):
    base = [10000.0 ** (-2 * i / 64) for i in range(32)]
    close = lambda a, b: all(abs(x - y) <= 1e-12 * abs(y) for x, y in zip(a, b))
    r = K.KdaRope.make(64, device="cpu")
    assert close(radians(r), base) and r.scale == 1.0 and not r.interleaved
    assert close(radians(K.KdaRope.make(64, scaling="linear", factor=4.0, device="cpu")), [f / 4 for f in base])
    n = radians(K.KdaRope.make(64, scaling="ntk", factor=4.0, interleaved=True, device="cpu"))
    assert n[0] == pytest.approx(1.0) and n[-1] == pytest.approx(base[-1] / 4)
    y = K.KdaRope.make(64, scaling="yarn", factor=8.0, original_len=4096, device="cpu")
    f = radians(y)
    assert y.scale == pytest.approx(0.1 * math.log(8.0) + 1.0)
    for a, b in zip(f, base):
        turns = 4096 * b / (2 * math.pi)
        assert b / 8 * 0.999999 <= a <= b * 1.000001
        if turns > 32 * 10000 ** (2 / 64):     # a whole pair above the border: kept
            assert a == pytest.approx(b)
        if turns < 10000 ** (-2 / 64):          # below the other: divided
            assert a == pytest.approx(b / 8)
    assert all(x > z for x, z in zip(f, f[1:]))
    for bad in (dict(rotary_dim=7), dict(rotary_dim=64, scaling="cubic"), dict(rotary_dim=64, factor=0.0), dict(rotary_dim=64, base=1.0),
                dict(rotary_dim=64, scaling="yarn", original_len=0), dict(rotary_dim=2, scaling="ntk")):
        with pytest.raises(ValueError):
            K.KdaRope.make(**bad, device="cpu")


def test_another_field_another_struct(K):
    r = K.KdaRope.make(32, device="cpu")
    st = r.c_struct()
    assert r.c_struct() is st and st.rotary_dim == 32
    r.turns = torch.zeros(8, dtype=torch.int64)
    r.interleaved = True
    assert r.c_struct().rotary_dim == 16 and r.c_struct().interleaved == 1
    r.turns = torch.zeros(8)
    with pytest.raises(TypeError):
        r.c_struct()
