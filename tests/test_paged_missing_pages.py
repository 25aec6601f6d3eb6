"""Page table entries that name no page where a key is needed: its tokens are left out of the sums, alike in
both attention calls, and the error word says so."""
from __future__ import annotations

import math

import pytest
import torch

from paged_ref import F64, check_attention, make_cache

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


def attention_without(q, k, v, length, scale, window, sinks, held):
    """paged_ref.attention where only the keys of `held` exist."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = torch.zeros(n, Hq, D, dtype=F64), torch.full((n, Hq), -math.inf, dtype=F64)
    mag, size = torch.zeros(n, Hq, D, dtype=F64), torch.zeros(n, Hq, dtype=F64)
    j = torch.arange(length)
    for t in range(n):
        p = length - n + t
        see = (j <= p) & held
        if window:
            see &= (j > p - window) | (j < sinks)
        if not see.any():
            continue
        kk, vv = k[see].repeat_interleave(G, 1), v[see].repeat_interleave(G, 1)
        s = torch.einsum("hd,jhd->hj", q[t], kk) * scale
        w = torch.softmax(s, 1)
        lse[t] = torch.logsumexp(s, 1)
        out[t] = torch.einsum("hj,jhd->hd", w, vv)
        mag[t] = torch.einsum("hj,jhd->hd", w, vv.abs())
        size[t] = (torch.einsum("hd,jhd->hj", q[t].abs(), kk.abs()) * scale).amax(1)
    return out, lse, mag, size


def run(K, lens, new, gone, Hkv, G, D, ps, dtype, kv, window, sinks, seed):
    """Rows of `lens` tokens without the pages `gone` [(row, page index, what the table says)], by prefill and by decode."""
    cache, dense = make_cache(K, lens, Hkv, D, ps, kv, seed)
    held = [torch.ones(n, dtype=torch.bool) for n in lens]
    for row, j, entry in gone:
        cache.page_table[row, j] = entry
        held[row][j * ps:(j + 1) * ps] = False
    B, scale = len(lens), D ** -0.5
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = (torch.randn(cu[-1], Hkv * G, D, generator=torch.Generator().manual_seed(seed + 1)) * 1.3).to(dtype)
    refs = [attention_without(q[cu[b]:cu[b + 1]].to(F64), *dense[b], lens[b], scale, window, sinks, held[b]) for b in range(B)]
    out, lse = K.kda_attn_prefill(cache, 0, i32(range(B)), i32(cu), max(new), q.cuda(), window=window, sinks=sinks, return_lse=True)
    assert K.kda_kv_get_error(cache) == 0x40
    for b in range(B):
        check_attention(out[cu[b]:cu[b + 1]], lse[cu[b]:cu[b + 1]], refs[b], dtype, lens[b])
    # the last tokens of each row by decode
    T = min(4, min(new))
    last = torch.stack([q[cu[b + 1] - T:cu[b + 1]] for b in range(B)])
    out, lse = K.kda_attn_decode(cache, 0, i32(range(B)), last.cuda(), window=window, sinks=sinks, return_lse=True)
    for b in range(B):
        check_attention(out[b], lse[b], [x[new[b] - T:] for x in refs[b]], dtype, lens[b])
    assert K.kda_kv_get_error(cache) in (0, 0x40)   # (decode's tokens need not see the missing pages)


@pytest.mark.parametrize("dtype,kv", TYPES, ids=IDS)
@pytest.mark.parametrize("D,ps", [(128, 64), (64, 16), (64, 128), (128, 32)])
def test_missing_pages(K, dtype, kv, D, ps):
    run(K, [300, 513, 129, 40], [140, 9, 129, 40], [(0, 0, -1), (1, 300 // ps, 1 << 30), (1, 513 // ps, -5), (2, 1, 10 ** 6)], 2, 3, D, ps, dtype, kv,
        0, 0, 71)


@pytest.mark.parametrize("dtype,kv", TYPES, ids=IDS)
def test_missing_pages_in_a_window_and_its_sinks(K, dtype, kv):
    run(K, [300, 700], [150, 20], [(0, 0, -1), (0, 12, -1), (1, 0, -1), (1, 41, 1 << 20), (1, 43, -1)], 1, 4, 64, 16, dtype, kv, 40, 19, 72)


def test_rows_whose_every_key_is_missing(K):
    """Nothing is left to see: 0 and -inf."""
    for dtype, kv in TYPES:
        run(K, [30, 20], [30, 5], [(0, 0, -1), (0, 1, -1), (1, 0, -1)], 1, 2, 64, 16, dtype, kv, 0, 0, 73)


def test_missing_pages_where_the_keys_are_split(K):
    run(K, [9000], [40], [(0, 0, -1), (0, 70, -1), (0, 139, 1 << 24)], 1, 4, 128, 64, BF, BF, 0, 0, 74)
    run(K, [5000], [3], [(0, 100, -1), (0, 101, -1)], 1, 2, 64, 32, BF, E4, 0, 0, 75)
