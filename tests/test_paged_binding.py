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
