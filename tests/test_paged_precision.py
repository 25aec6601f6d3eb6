"""Where the weights' sixteen bits could lose what counts: many small ones behind a few large ones."""
from __future__ import annotations

import pytest
import torch

from paged_ref import EPS, F64, check_attention

pytestmark = pytest.mark.gpu

BF, FH, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
TYPES = [(BF, BF), (FH, FH), (BF, E4), (FH, E4)]
IDS = ["bf16", "fp16", "bf16-e4m3", "fp16-e4m3"]


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def shared_cache(K, k, v, ps, rows, dtype, scale=1.0):
    """`rows` rows that hold the same tokens (k, v [N, D]) in the same pages."""
    N, D = k.shape
    n = -(-N // ps)
    pad = lambda x: torch.cat([x, x.new_zeros(n * ps - N, D)]).view(1, n, 1, ps, D).to(dtype).cuda()
    fp8 = dtype == E4
    sc = torch.full((1, 1), scale, device="cuda") if fp8 else None
    return K.KdaKvCache(k=pad(k / scale if fp8 else k), v=pad(v / scale if fp8 else v),
                        page_table=torch.arange(n, dtype=torch.int32, device="cuda")[None].expand(rows, n).contiguous(),
                        seq_lens=torch.full((rows,), N, dtype=torch.int32, device="cuda"),
                        page_refs=torch.full((n,), rows, dtype=torch.int32, device="cuda"), k_scale=sc, v_scale=sc)


def tail(N, D, dtype, nats, seed):
    """Four sinks (one for each 16 of the first 64 keys) whose scores are `nats` above all others' and whose values are 0; the
    others' values are around one.  A query of (1, 0, ...) and a scale of 1 give these scores, exactly (codes of
    8 bits stand for 1/64 of `nats`)."""
    scale = nats / 64
    g = torch.Generator().manual_seed(seed)
    k = torch.zeros(N, D)
    k[0:64:16, 0] = nats
    v = 1 + 0.2 * torch.randn(N, D, generator=g)
    v[0:64:16] = 0
    q8 = lambda x: ((x / scale).to(E4).float() * scale) if dtype == E4 else x.to(dtype).float()
    return q8(k), q8(v)


def expect(k, v, upto):
    """out, lse, mag, size of a query (1, 0, ...) over the first `upto` keys, as paged_ref.attention gives them."""
    s = k[:upto, 0].to(F64)
    w = torch.softmax(s, 0)
    x = v[:upto].to(F64)
    return (w @ x)[None, None], torch.logsumexp(s, 0)[None, None], (w @ x.abs())[None, None], s.abs().max()[None, None]


# 17.25 nats are 24.9 powers of two
@pytest.mark.parametrize("dtype,kv", TYPES, ids=IDS)
def test_many_small_weights_behind_sinks_in_prefill(K, dtype, kv):
    """2500 tokens of 8 heads: enough row tiles that the keys are not split."""
    D, ps, n, G = 64, 128, 2500, 8
    for N in (32768, 131072):
        k, v = tail(N, D, kv, 17.25, 81)
        cache = shared_cache(K, k, v, ps, 1, kv, 17.25 / 64)
        q = torch.zeros(n, G, D, dtype=dtype, device="cuda")
        q[..., 0] = 1
        out, lse = K.kda_attn_prefill(cache, 0, i32([0]), i32([0, n]), n, q, scale=1.0, return_lse=True)
        assert K.kda_kv_get_error(cache) == 0
        for t in (0, 1234, n - 1):
            out_, lse_, mag, size = expect(k, v, N - n + t + 1)
            check_attention(out[t:t + 1], lse[t:t + 1], (out_.expand(1, G, D), lse_.expand(1, G), mag.expand(1, G, D), size.expand(1, G)), dtype, N)


@pytest.mark.parametrize("dtype,kv", TYPES, ids=IDS)
@pytest.mark.parametrize("T,G", [(1, 4), (3, 5), (4, 8)])
def test_many_small_weights_behind_sinks_in_decode(K, dtype, kv, T, G):
    """More rows than CTAs, so that a CTA holds a whole row; each of its warps has a sink."""
    D, ps, N, rows = 64, 128, 32768, 700
    k, v = tail(N, D, kv, 17.25, 82)
    cache = shared_cache(K, k, v, ps, rows, kv, 17.25 / 64)
    q = torch.zeros(rows, T, G, D, dtype=dtype, device="cuda")
    q[..., 0] = 1
    out, lse = K.kda_attn_decode(cache, 0, i32(range(rows)), q, scale=1.0, return_lse=True)
    assert K.kda_kv_get_error(cache) == 0
    for t in range(T):
        out_, lse_, mag, size = expect(k, v, N - T + t + 1)
        for b in (0, 333, rows - 1):
            check_attention(out[b, t:t + 1], lse[b, t:t + 1], (out_.expand(1, G, D), lse_.expand(1, G), mag.expand(1, G, D), size.expand(1, G)), dtype, N)


@pytest.mark.parametrize("dtype,kv", TYPES[1:], ids=IDS[1:])
def test_weights_under_the_normal_range(K, dtype, kv):
    """22 nats (31.7 powers of two) below: weights that are halves' subnormals lose at most 2^-25 of a P that stands at 2^11
    for the largest key at least: 2^-36 of that key's weight each."""
    D, ps, n, G, N = 64, 128, 2500, 8, 32768
    k, v = tail(N, D, kv, 22.0, 83)
    cache = shared_cache(K, k, v, ps, 1, kv, 22.0 / 64)
    q = torch.zeros(n, G, D, dtype=dtype, device="cuda")
    q[..., 0] = 1
    out, lse = K.kda_attn_prefill(cache, 0, i32([0]), i32([0, n]), n, q, scale=1.0, return_lse=True)
    want, _, mag, size = expect(k, v, N)
    s_err, l_err = D * 2.0 ** -23 * size[..., None] + 2.0 ** -20, N * 2.0 ** -24 + 2.0 ** -20   # as in check_attention
    tol = 1.01 * (EPS[dtype] * (want.abs() + mag) + 2 * (s_err + l_err) * mag) + N * 2.0 ** -36 * v.abs().max() + 2.0 ** -24
    assert ((out[-1:].to(F64).cpu() - want).abs() <= tol).all()
