"""Offsets that go back and forth: sequences that share tokens do no harm."""
from __future__ import annotations

import pytest
import torch

from paged_ref import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def test_offsets_that_name_the_same_tokens_many_times(K):
    """Every third sequence is the whole prompt: more row tiles than the tokens can have.  The call is left out, and the
    next one finds its workspace ready."""
    N, G, B = 512, 4, 700
    cache, _ = make_cache(K, [600], 1, 64, 16, torch.bfloat16, 91)
    q = torch.randn(N, G, 64, generator=torch.Generator().manual_seed(92)).to(torch.bfloat16).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ref = K.kda_attn_prefill(cache, 0, i32([0]), i32([0, N]), N, q)
    assert K.kda_kv_get_error(cache) == 0
    for n in (300, B):   # all within the table that is kept on chip, and past it
        out = torch.full_like(ref, 5.0)
        K.kda_attn_prefill(cache, 0, i32([0] * n), i32([(0, 0, N)[i % 3] for i in range(n + 1)]), N, q, out=out)
        assert K.kda_kv_get_error(cache) == 0x20
        assert (out == 5).all()
        assert torch.equal(K.kda_attn_prefill(cache, 0, i32([0]), i32([0, N]), N, q), ref)
    assert K.kda_kv_get_error(cache) == 0
