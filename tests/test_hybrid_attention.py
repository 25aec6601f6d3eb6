"""examples/hybrid_decode.py: each attention call of the served model against the formula on what its cache holds.

(The example's own comparison is of whole outputs, in which an E4M3 cache's steps leave wide room.)"""
from __future__ import annotations

import os
import sys

import pytest
import torch

from paged_ref import F64, attention, check_attention

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def E():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import hybrid_decode as E
    finally:
        sys.path.pop(0)
    return E


def dense(cache, layer, row):
    """Keys, values [len, Hkv, D] in 64 bits of a row."""
    n, ps = int(cache.seq_lens[row]), cache.k.shape[3]
    pages = cache.page_table[row, :-(-n // ps)].long()
    got = []
    for x, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        y = x[layer].view(torch.uint8 if sc is not None else x.dtype)[pages].view(x.dtype).cpu().to(F64).transpose(1, 2).flatten(0, 1)[:n]
        got.append(y if sc is None else y * sc[layer].to(F64).cpu()[:, None])
    return got


def check(out, q, cache, layer, row, window=0, sinks=0):
    n = int(cache.seq_lens[row])
    check_attention(out, None, attention(q.cpu().to(F64), *dense(cache, layer, row), n, q.shape[-1] ** -0.5, window, sinks), q.dtype, n)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])
def test_every_attention_call_of_the_served_model(E, dtype, monkeypatch):
    K, calls = E.K, {"decode": 0, "prefill": 0}
    decode, prefill = K.kda_attn_decode, K.kda_attn_prefill

    def checked_decode(cache, layer, rows, q, **kw):
        out = decode(cache, layer, rows, q, **kw)
        for b, row in enumerate(rows.tolist()):
            check(out[b], q[b], cache, layer, row, **kw)
        calls["decode"] += 1
        return out

    def checked_prefill(cache, layer, rows, cu, most, q, **kw):
        out = prefill(cache, layer, rows, cu, most, q, **kw)
        for b, row in enumerate(rows.tolist()):
            check(out[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], cache, layer, row, **kw)
        calls["prefill"] += 1
        return out

    monkeypatch.setattr(K, "kda_attn_decode", checked_decode)
    monkeypatch.setattr(K, "kda_attn_prefill", checked_prefill)
    E.serve(E.Hybrid(cache_dtype=dtype))
    assert calls["decode"] >= 16 and calls["prefill"] >= 4   # two attention layers: 8 steps, 2 prompts
    # and a layer that gave zeros would not pass
    monkeypatch.setattr(K, "kda_attn_decode", lambda *a, **kw: (checked_decode(*a, **kw), check(torch.zeros_like(a[3][0]), a[3][0], a[0], a[1], int(a[2][0]), **kw))[0])
    with pytest.raises(AssertionError, match="tolerance"):
        E.serve(E.Hybrid(cache_dtype=dtype))
