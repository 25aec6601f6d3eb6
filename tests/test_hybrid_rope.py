"""examples/hybrid_decode.py with rotated positions and a 4-bit cache: each rotation against complex products, each attention
call of the served model against the formula on what its cache holds."""
from __future__ import annotations

import math
import os
import sys

import pytest
import torch

from codes_ref import turn_error, turned, unpacked, values
from paged_ref import EPS, F64, attention, check_attention

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
    n = int(cache.seq_lens[row])
    pages = cache.page_table[row, :-(-n // cache.k.shape[3])].long()
    got = []
    for x, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        if cache.k.dtype == torch.uint8:
            codes, s = unpacked(x[layer, pages].cpu(), cache.head_dim)
            y = values(codes, s, 1.0) * sc[layer].cpu().to(F64)[:, None, None]
        else:
            y = x[layer, pages].cpu().to(F64)
        got.append(y.transpose(1, 2).flatten(0, 1)[:n])
    return got


@pytest.mark.parametrize("dtype,rotary", [(torch.bfloat16, 32), (torch.uint8, 64)], ids=["bf16-half", "e2m1"])
def test_every_call_of_the_served_model(E, dtype, rotary, monkeypatch):
    K, calls = E.K, {"append": 0, "decode": 0, "prefill": 0}
    append, decode, prefill = K.kda_kv_append_rope, K.kda_attn_decode, K.kda_attn_prefill
    model = E.Hybrid(cache_dtype=dtype, rotary_dim=rotary)
    freqs = [math.ldexp(float(t % 2 ** 64), -64) * 2 * math.pi for t in model.rope.turns.tolist()]

    def checked_append(cache, layer, rows, rope, q, k, v, cu_seqlens=None):
        out = append(cache, layer, rows, rope, q, k, v, cu_seqlens=cu_seqlens)
        for b, row in enumerate(rows.tolist()):
            x, y = (t[cu_seqlens[b]:cu_seqlens[b + 1]].cpu() if cu_seqlens is not None else t[b].cpu() for t in (q, out))
            n = int(cache.seq_lens[row])
            pos = torch.arange(n - x.shape[0], n)
            ref, err = turned(x, pos, freqs, scale=rope.scale), turn_error(x, rotary, scale=rope.scale)
            assert ((y.to(F64) - ref).abs() <= 1.001 * EPS[torch.bfloat16] * (ref.abs() + err) + err).all()
        calls["append"] += 1
        return out

    def check(out, q, cache, layer, row, window=0, sinks=0):
        n = int(cache.seq_lens[row])
        check_attention(out, None, attention(q.cpu().to(F64), *dense(cache, layer, row), n, q.shape[-1] ** -0.5, window, sinks), q.dtype, n)

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

    monkeypatch.setattr(K, "kda_kv_append_rope", checked_append)
    monkeypatch.setattr(K, "kda_attn_decode", checked_decode)
    monkeypatch.setattr(K, "kda_attn_prefill", checked_prefill)
    worst = E.serve(model)
    assert calls["decode"] >= 16 and calls["prefill"] >= 4 and calls["append"] == calls["decode"] + calls["prefill"]
    if dtype == torch.bfloat16:   # the steps and the prompt round alike (see test_hybrid_example.py)
        assert worst <= 4 * 3 * 2 * 2.0 ** -8 + 2 * 2 * 2 * 2.0 ** -8   # ... and the two attention layers' rotated q and k
