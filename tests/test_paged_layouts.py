"""Prefill queries in the layouts that callers have them in: any strides of tokens and heads."""
from __future__ import annotations

import pytest
import torch

from paged_ref import F64, attention, check_attention, make_cache

pytestmark = pytest.mark.gpu

BF, FH, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
N, D = 150, 64


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def strided(q, token, head):
    """q [N, H, D] held with these strides (elements)."""
    flat = torch.full(((q.shape[0] - 1) * token + (q.shape[1] - 1) * head + D,), 9.0, dtype=q.dtype, device="cuda")
    x = flat.as_strided(q.shape, (token, head, 1))
    x.copy_(q)
    return x


LAYOUTS = {
    "head-major": lambda q: q.transpose(0, 1).contiguous().transpose(0, 1),
    "padded heads": lambda q: strided(q, q.shape[1] * 72, 72),
    "padded heads and tokens": lambda q: strided(q, q.shape[1] * 72 + 8, 72),
    "heads apart, tokens between them": lambda q: strided(q, 72, N * 72 + 8),
    "every other token": lambda q: strided(q, 2 * q.shape[1] * D, D),
    "tokens apart by no multiple of a head": lambda q: strided(q, q.shape[1] * D + 40, D),
}


@pytest.mark.parametrize("dtype,kv", [(BF, BF), (FH, FH), (BF, E4), (FH, E4)], ids=["bf16", "fp16", "bf16-e4m3", "fp16-e4m3"])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 4), (1, 3), (1, 8)])
@pytest.mark.parametrize("name", LAYOUTS)
def test_query_layouts(K, dtype, kv, Hkv, G, name):
    cache, dense = make_cache(K, [170, 90], Hkv, D, 16, kv, 95)
    q = (torch.randn(N, Hkv * G, D, generator=torch.Generator().manual_seed(96)) * 1.3).to(dtype)
    x = LAYOUTS[name](q.cuda())
    assert torch.equal(x.cpu(), q)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    out, lse = K.kda_attn_prefill(cache, 0, i32([0, 1]), i32([0, 101, N]), 101, x, return_lse=True)
    assert K.kda_kv_get_error(cache) == 0
    for a, b, row, n in ((0, 101, 0, 170), (101, N, 1, 90)):
        check_attention(out[a:b], lse[a:b], attention(q[a:b].to(F64), *dense[row], n, D ** -0.5, 0, 0), dtype, n)


@pytest.mark.parametrize("dtype,kv", [(BF, BF), (BF, E4)], ids=["bf16", "bf16-e4m3"])
def test_broadcast_queries(K, dtype, kv):
    """One head's queries for all heads, one token's for all tokens."""
    cache, dense = make_cache(K, [N], 2, D, 16, kv, 97)
    g = torch.Generator().manual_seed(98)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for q in (torch.randn(N, 1, D, generator=g).to(dtype).expand(N, 8, D), torch.randn(1, 8, D, generator=g).to(dtype).expand(N, 8, D)):
        x = q[:1].cuda().expand(N, 8, D) if q.stride(0) == 0 else q[:, :1].cuda().expand(N, 8, D)
        out, lse = K.kda_attn_prefill(cache, 0, i32([0]), i32([0, N]), N, x, return_lse=True)
        check_attention(out, lse, attention(q.to(F64), *dense[0], N, D ** -0.5, 0, 0), dtype, N)
