"""Key scales and softmax scales outside the usual: NaN, and zero with the largest queries."""
from __future__ import annotations

import math

import pytest
import torch

from paged_ref import F64, check_attention

pytestmark = pytest.mark.gpu

BF, FH, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF, FH], ids=["bf16", "fp16"])
def test_a_scale_that_is_no_number_shows(K, dtype):
    """A NaN in a layer's key scale makes that head's outputs NaN, not an average, and leaves the other head's alone."""
    g = torch.Generator().manual_seed(84)
    kv = torch.randn(1, 4, 2, 16, 64, generator=g).to(E4).cuda()
    cache = K.KdaKvCache(k=kv, v=kv.clone(), page_table=i32([[0, 1, 2, 3]]), seq_lens=i32([60]), page_refs=i32([1, 1, 1, 1]),
                         k_scale=torch.tensor([[math.nan, 0.5]], device="cuda"), v_scale=torch.ones(1, 2, device="cuda"))
    q = torch.randn(40, 4, 64, generator=g).to(dtype).cuda()
    a, la = K.kda_attn_prefill(cache, 0, i32([0]), i32([0, 40]), 40, q, return_lse=True)
    for T in (1, 4):   # two and eight rows a block
        b, lb = K.kda_attn_decode(cache, 0, i32([0]), q[None, -T:], return_lse=True)
        assert b[:, :, :2].isnan().all() and lb[:, :, :2].isnan().all()
        assert not b[:, :, 2:].isnan().any() and not lb[:, :, 2:].isnan().any()
    assert a[:, :2].isnan().all() and la[:, :2].isnan().all()
    assert not a[:, 2:].isnan().any() and not la[:, 2:].isnan().any()


def test_a_scale_of_zero_with_the_largest_queries(K):
    """Scores of 0 whatever the queries: the average of the values, log of their number."""
    g = torch.Generator().manual_seed(85)
    kv = torch.randn(1, 4, 1, 16, 64, generator=g).to(E4).cuda()
    ones = torch.ones(1, 1, device="cuda")
    cache = K.KdaKvCache(k=kv, v=kv.clone(), page_table=i32([[0, 1, 2, 3]]), seq_lens=i32([60]), page_refs=i32([1, 1, 1, 1]), k_scale=ones, v_scale=ones)
    q = (torch.randn(3, 2, 64, generator=g) * 1e38).clamp(-3e38, 3e38).to(BF).cuda()
    dense = kv.float().cpu()[0, :, 0].reshape(64, 64).to(F64)
    a, la = K.kda_attn_prefill(cache, 0, i32([0]), i32([0, 3]), 3, q, scale=0.0, return_lse=True)
    b, lb = K.kda_attn_decode(cache, 0, i32([0]), q[None], scale=0.0, return_lse=True)
    for t in range(3):
        x = dense[:58 + t]
        ref = (x.mean(0)[None, None].expand(1, 2, 64), torch.full((1, 2), math.log(58 + t), dtype=F64),
               x.abs().mean(0)[None, None].expand(1, 2, 64), torch.zeros(1, 2, dtype=F64))
        check_attention(a[t:t + 1], la[t:t + 1], ref, BF, 60)
        check_attention(b[0, t:t + 1], lb[0, t:t + 1], ref, BF, 60)
