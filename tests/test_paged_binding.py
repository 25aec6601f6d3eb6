"""What the paged binding keeps between calls, and what it hands on (no GPU needed)."""
from __future__ import annotations

import pytest
import torch


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def cpu_cache(K, **kw):
    d = dict(layers=1, num_pages=4, Hkv=2, rows=2, max_pages=2, page_size=16, head_dim=64, device="cpu")
    d.update(kw)
    return K.KdaKvCache.zeros(**d)


def test_numbers_in_tensors_are_read_at_every_call(K):
    """A scale, a window or sinks may be 0-dim tensors: a value that changes in place counts from the next call on."""
    c = cpu_cache(K)
    c.c_struct()
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    scale, window, sinks = torch.tensor(0.5), torch.tensor(8), torch.tensor(2)
    for s, w, n in ((0.5, 8, 2), (2.0, 8, 2), (2.0, 30, 2), (2.0, 30, 5), (0.5, 8, 2)):
        scale.fill_(s)
        window.fill_(w)
        sinks.fill_(n)
        desc = K.paged._attn(c, q, False, scale, window, sinks, None, None, False)[0]._obj
        assert (desc.scale, desc.window, desc.sinks) == (s, w, n)
    assert len(c.__dict__["_plans"]) == 4   # by value: the last one is the first again


@pytest.mark.parametrize("bits,cleared", [(0x4, True), (0x44, True), (0x40, False), (0, False)])
def test_a_wait_that_gave_up_clears_the_own_workspace(K, monkeypatch, bits, cleared):
    """Counters may be left above 0 by a call that ended so; reading its error makes the cache ready again."""
    import contextlib

    class Fake:
        @staticmethod
        def kda_kv_get_error(cache, host, stream):
            host._obj.value = bits
            return K.kda.KDA_ERR_DEVICE if bits else 0

        kda_kv_workspace_size = K.library().kda_kv_workspace_size
        kda_attn_workspace_size = K.library().kda_attn_workspace_size

    c = cpu_cache(K)
    c.c_struct()
    c.__dict__["_attn_ws"][:64] = 1
    monkeypatch.setattr(K.paged, "_lib", Fake)
    monkeypatch.setattr(K.paged, "_stream", lambda stream, dev: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    assert K.kda_kv_get_error(c) == bits
    assert bool(c.__dict__["_attn_ws"].any()) != cleared
