"""The paged cache's C entry points and their binding (no GPU needed): every argument is checked on the
host before anything is launched.  All calls below fail those checks or are documented no-ops, so no
kernel ever sees the fake pointers."""
from __future__ import annotations

import ctypes

import pytest
import torch

P = 0x10000   # a fake, aligned device pointer


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def cache(K, **kw):
    d = dict(k=P, v=P, kv_dtype=0, num_layers=2, num_pages=8, num_kv_heads=2, page_size=16, head_dim=64, rows=4,
             max_pages=4, page_table=P, seq_lens=P, page_refs=P, k_scale=None, v_scale=None, err_word=P)
    d.update(kw)
    return K.paged._Cache(**d)


def layout(K, **kw):
    d = dict(dtype=0, seq_stride=128, token_stride=128, head_stride=64)
    d.update(kw)
    return K.paged._Layout(**d)


def desc(K, **kw):
    d = dict(num_q_heads=4, scale=0.125, window=0, sinks=0, q=layout(K))
    d.update(kw)
    return K.paged._Desc(**d)


def ref(x):
    return None if x is None else ctypes.byref(x)


def extend(K, c, rows=P, n=None, n_all=1, B=1, ws=P, size=1 << 20):
    return K.library().kda_kv_extend(ref(c), rows, n, n_all, B, ws, size, None)


def append(K, c, layer=0, rows=P, B=1, T=1, n=None, cu=None, k=P, kl=None, v=P, vl=None):
    kl, vl = layout(K) if kl is None else kl, layout(K) if vl is None else vl
    return K.library().kda_kv_append(ref(c), layer, rows, B, T, n, cu, k, ref(kl), v, ref(vl), None)


def decode(K, c, layer=0, d=None, rows=P, B=1, T=1, n=None, q=P, out=P, lse=None, ws=P, size=1 << 40):
    d = desc(K) if d is None else d
    return K.library().kda_attn_decode(ref(c), layer, ref(d), rows, B, T, n, q, out, lse, ws, size, None)


def prefill(K, c, layer=0, d=None, rows=P, B=1, cu=P, total=1, most=1, q=P, out=P, lse=None, ws=P, size=1 << 40):
    d = desc(K) if d is None else d
    return K.library().kda_attn_prefill(ref(c), layer, ref(d), rows, B, cu, total, most, q, out, lse, ws, size, None)


def msg(K):
    return K.library().kda_last_error().decode()


BAD_CACHES = [(dict(kv_dtype=3), "kv_dtype", 1), (dict(num_layers=0), "num_layers", 1), (dict(num_pages=0), "num_pages", 1),
              (dict(num_kv_heads=0), "num_kv_heads", 1), (dict(num_kv_heads=5000), "num_kv_heads", 1),
              (dict(rows=0), "rows", 1), (dict(max_pages=0), "max_pages", 1), (dict(page_size=48), "page_size", 2),
              (dict(head_dim=96), "head_dim", 2), (dict(rows=(1 << 18) + 1), "rows", 2),
              (dict(rows=1 << 18, max_pages=1 << 14), "31 bits", 2), (dict(max_pages=1 << 28), "tokens", 2),
              (dict(num_pages=1 << 30), "num_pages", 2), (dict(k=None), "k is null", 1), (dict(v=P + 8), "16-byte", 1),
              (dict(page_table=P + 2), "page_table", 1), (dict(seq_lens=None), "seq_lens", 1), (dict(page_refs=None), "page_refs", 1),
              (dict(err_word=None), "err_word", 1), (dict(kv_dtype=2), "k_scale", 1), (dict(kv_dtype=2, k_scale=P), "v_scale", 1)]


@pytest.mark.parametrize("kw,word,status", BAD_CACHES, ids=lambda x: str(x)[:40])
def test_every_entry_checks_the_cache(K, kw, word, status):
    lib = K.library()
    c = cache(K, **kw)
    for call in (lambda: extend(K, c), lambda: lib.kda_kv_truncate(ref(c), P, P, 1, P, 1 << 40, None),
                 lambda: lib.kda_kv_fork(ref(c), P, P, 1, P, 1 << 40, None), lambda: lib.kda_kv_compact(ref(c), P, P, 1 << 40, None),
                 lambda: append(K, c), lambda: decode(K, c), lambda: prefill(K, c)):
        assert call() == status
        assert word in msg(K)


def test_null_structs(K):
    lib = K.library()
    assert extend(K, None) == 1 and "cache" in msg(K)
    c = cache(K)
    assert lib.kda_attn_decode(ref(c), 0, None, P, 1, 1, None, P, P, None, P, 1 << 40, None) == 1 and "desc" in msg(K)
    assert lib.kda_kv_append(ref(c), 0, P, 1, 1, None, None, P, None, P, None, None) == 1 and "layout of k" in msg(K)
    assert lib.kda_kv_get_error(None, None, None) == 1
    assert lib.kda_kv_workspace_size(None) == 0 and lib.kda_attn_workspace_size(None) == 0


def test_page_calls_check_their_arguments(K):
    lib, c = K.library(), cache(K)
    assert extend(K, c, B=-1) == 1 and extend(K, c, B=5) == 1 and "distinct" in msg(K)
    assert extend(K, c, n_all=-1) == 1 and "n_all" in msg(K)
    assert extend(K, c, rows=None) == 1 and extend(K, c, n=P + 1) == 1
    assert extend(K, c, ws=None) == 1 and extend(K, c, ws=P + 16) == 1 and "256" in msg(K)
    need = lib.kda_kv_workspace_size(ref(c))
    assert need > 0 and extend(K, c, size=need - 1) == 1 and "workspace_bytes" in msg(K)
    assert lib.kda_kv_truncate(ref(c), P, None, 1, P, need, None) == 1 and "new_lens" in msg(K)
    assert lib.kda_kv_fork(ref(c), None, P, 1, P, need, None) == 1 and "src_rows" in msg(K)
    assert lib.kda_kv_compact(ref(c), None, P, need, None) == 1 and "remap" in msg(K)
    # nothing to do: nothing is launched
    assert extend(K, c, B=0, rows=None, ws=None) == 0
    assert lib.kda_kv_truncate(ref(c), None, None, 0, None, 0, None) == 0
    assert lib.kda_kv_fork(ref(c), None, None, 0, None, 0, None) == 0


def test_append_checks_its_arguments(K):
    c, c8 = cache(K), cache(K, kv_dtype=2, k_scale=P, v_scale=P)
    for layer in (-1, 2):
        assert append(K, c, layer=layer) == 1 and "layer" in msg(K)
    assert append(K, c, B=-1) == 1 and append(K, c, T=-1) == 1
    assert append(K, c, kl=layout(K, dtype=2)) == 1 and "dtype" in msg(K)
    assert append(K, c, kl=layout(K, dtype=1), vl=layout(K, dtype=1)) == 1 and "cache holds" in msg(K)
    assert append(K, c8, kl=layout(K, dtype=1)) == 1 and "different types" in msg(K)
    assert append(K, c, kl=layout(K, head_stride=60)) == 1 and "multiples of 8" in msg(K)
    assert append(K, c, vl=layout(K, token_stride=-128)) == 1 and "negative" in msg(K)
    assert append(K, c, n=P, cu=P) == 1 and "exclude" in msg(K)
    assert append(K, c, B=1 << 20, T=1 << 12) == 2 and "31 bits" in msg(K)
    assert append(K, c, k=P + 8) == 1 and append(K, c, v=None) == 1 and append(K, c, rows=None) == 1 and append(K, c, cu=P + 1) == 1
    assert append(K, c, B=0) == 0 and append(K, c, T=0) == 0


def test_attention_checks_its_arguments(K):
    lib, c = K.library(), cache(K)
    for call in (decode, prefill):
        assert call(K, c, layer=2) == 1 and "layer" in msg(K)
        assert call(K, c, d=desc(K, num_q_heads=3)) == 1 and "multiple" in msg(K)
        assert call(K, c, d=desc(K, num_q_heads=130)) == 2 and "64 per kv head" in msg(K)
        for scale in (float("nan"), float("inf"), -1.0):
            assert call(K, c, d=desc(K, scale=scale)) == 1 and "scale" in msg(K)
        assert call(K, c, d=desc(K, window=-1)) == 1 and call(K, c, d=desc(K, sinks=-1)) == 1 and "sinks" in msg(K)
        assert call(K, c, d=desc(K, q=layout(K, dtype=1))) == 1 and "cache holds" in msg(K)
        assert call(K, c, B=-1) == 1 and call(K, c, B=65536) == 2
        assert call(K, c, rows=None) == 1 and call(K, c, q=P + 8) == 1 and call(K, c, out=None) == 1 and call(K, c, lse=P + 2) == 1
        assert call(K, c, ws=None) == 1 and call(K, c, ws=P + 64) == 1
        need = lib.kda_attn_workspace_size(ref(c))
        assert need > 0 and call(K, c, size=need - 1) == 1 and "workspace_bytes" in msg(K)
        assert call(K, c, B=0) == 0
    for T in (0, 17):
        assert decode(K, c, T=T) == 1 and "T=" in msg(K)
    assert decode(K, c, n=P + 2) == 1
    assert prefill(K, c, total=-1) == 1 and prefill(K, c, most=-1) == 1 and prefill(K, c, most=0) == 1 and prefill(K, c, cu=None) == 1
    assert prefill(K, c, total=1 << 30, d=desc(K, num_q_heads=8)) == 2 and "rows" in msg(K)
    assert prefill(K, c, total=0) == 0


def cpu_cache(K, **kw):
    d = dict(layers=1, num_pages=4, Hkv=2, rows=2, max_pages=2, page_size=16, head_dim=64, device="cpu")
    d.update(kw)
    return K.KdaKvCache.zeros(**d)


def test_binding_checks_tensors(K):
    i32 = torch.int32
    rows = torch.zeros(1, dtype=i32)
    with pytest.raises(TypeError):
        K.KdaKvCache(torch.zeros(1, 2, 2, 16, 64), torch.zeros(1, 2, 2, 16, 64), torch.zeros(1, 2, dtype=i32),
                     torch.zeros(1, dtype=i32), torch.zeros(2, dtype=i32)).c_struct()
    c = cpu_cache(K)
    c.seq_lens = torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError):
        c.c_struct()
    c = cpu_cache(K, dtype=torch.float8_e4m3fn)
    assert c.c_struct().kv_dtype == 2
    c.v_scale = None
    with pytest.raises(ValueError):
        c.c_struct()
    c = cpu_cache(K)
    st = c.c_struct()
    assert c.c_struct() is st and (st.page_size, st.head_dim, st.rows, st.max_pages) == (16, 64, 2, 2)
    c.page_table = torch.zeros(5, 7, dtype=i32)   # another tensor: another struct, with its sizes
    c.seq_lens = torch.zeros(5, dtype=i32)
    assert (c.c_struct().rows, c.c_struct().max_pages) == (5, 7)
    c = cpu_cache(K)
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    for bad in (torch.zeros(1, 2, dtype=i32), torch.zeros(1), [0]):
        with pytest.raises((ValueError, TypeError)):
            K.kda_attn_decode(c, 0, bad, q)
    for bad in (q.float(), q.half()):
        with pytest.raises(TypeError):
            K.kda_attn_decode(c, 0, rows, bad)
    with pytest.raises(ValueError):
        K.kda_attn_decode(c, 0, rows, torch.zeros(1, 1, 4, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        K.kda_attn_decode(c, 0, rows, torch.zeros(1, 1, 64, 4, dtype=torch.bfloat16).transpose(2, 3))
    with pytest.raises(ValueError):
        K.kda_attn_decode(c, 0, rows, torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        K.kda_attn_decode(c, 0, rows, q, out=q.float())
    with pytest.raises(ValueError):
        K.kda_attn_prefill(c, 0, rows, torch.zeros(3, dtype=i32), 1, q[0])
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        K.kda_kv_append(c, 0, torch.zeros(2, dtype=i32), k, k)   # 3 tokens, 2 rows, no offsets
    with pytest.raises(ValueError):
        K.kda_kv_append(c, 0, rows, k, k[:2])
    with pytest.raises(ValueError):
        K.kda_kv_append(c, 0, rows, k[None], k[None], cu_seqlens=torch.zeros(2, dtype=i32))
    with pytest.raises(TypeError):
        K.kda_kv_extend(c, rows, torch.zeros(1))


def test_binding_refuses_numbers_past_32_bits(K):
    """2^32 + 1 does not arrive as 1."""
    c, i32, past = cpu_cache(K), torch.int32, (1 << 32) + 1
    rows, cu = torch.zeros(1, dtype=i32), torch.zeros(2, dtype=i32)
    q, k = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    many = k[0, :1].expand(past, 2, 64)   # no memory behind it
    for call in (lambda: K.kda_kv_extend(c, rows, past), lambda: K.kda_kv_append(c, past, rows, k, k),
                 lambda: K.kda_kv_append(c, 0, rows, many, many, cu_seqlens=cu),
                 lambda: K.kda_attn_decode(c, past, rows, q), lambda: K.kda_attn_decode(c, 0, rows, q, window=past),
                 lambda: K.kda_attn_decode(c, 0, rows, q, window=4, sinks=past),
                 lambda: K.kda_attn_prefill(c, past, rows, cu, 1, q[0]), lambda: K.kda_attn_prefill(c, 0, rows, cu, past, q[0])):
        with pytest.raises(ValueError, match="32 bits"):
            call()
