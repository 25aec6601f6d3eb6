"""A paged cache's own workspaces: made and cleared with the cache, before any stream or graph can use them."""
from __future__ import annotations

import pytest
import torch

from paged_ref import F64, attention, check_attention, make_cache

BF = torch.bfloat16


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def cpu_cache(K, **kw):
    d = dict(layers=1, num_pages=4, Hkv=2, rows=2, max_pages=2, page_size=16, head_dim=64, device="cpu")
    d.update(kw)
    return K.KdaKvCache.zeros(**d)


def owned(cache):
    return {k: cache._workspace(k, None) for k in ("_kv_ws", "_attn_ws")}


def test_workspaces_are_made_with_the_cache(K, monkeypatch):
    c = cpu_cache(K)
    need = K.kda_attn_workspace_size(c), K.kda_kv_workspace_size(c)
    monkeypatch.setattr(torch, "zeros", None)   # no call makes or clears one
    monkeypatch.setattr(torch, "empty", None)
    got = owned(c)
    assert got["_attn_ws"][1] >= need[0] and got["_kv_ws"][1] >= need[1]
    assert not c.__dict__["_attn_ws"].any()
    assert owned(c) == got


def test_a_field_that_changes_keeps_workspaces_that_still_fit(K):
    c = cpu_cache(K)
    c.c_struct()
    before = owned(c)
    c.seq_lens = torch.zeros(2, dtype=torch.int32)
    c.c_struct()
    assert owned(c) == before
    c.page_table, c.seq_lens = torch.zeros(500, 7, dtype=torch.int32), torch.zeros(500, dtype=torch.int32)
    c.c_struct()
    assert owned(c)["_attn_ws"] == before["_attn_ws"]            # its size does not depend on the rows
    assert owned(c)["_kv_ws"][1] >= K.kda_kv_workspace_size(c) > before["_kv_ws"][1]


def test_no_workspace_is_made_inside_a_capture(K, monkeypatch):
    """A cache made while a graph is captured has none (its clear would only run with the graph): its calls ask
    for one."""
    monkeypatch.setattr(K.paged, "_capturing", lambda dev: True)
    c = cpu_cache(K)
    for kind in ("_kv_ws", "_attn_ws"):
        with pytest.raises(RuntimeError, match="captur"):
            c._workspace(kind, None)
    mine = torch.zeros(1 << 20, dtype=torch.uint8)
    assert c._workspace("_attn_ws", mine) == (mine.data_ptr(), 1 << 20)
    monkeypatch.setattr(K.paged, "_capturing", lambda dev: False)
    assert owned(c)["_attn_ws"][1] >= K.kda_attn_workspace_size(c)   # afterwards it has


# ---------------------------------------------------------------- on the GPU

LENS = [3000, 17, 700, 1]


def dirty_blocks(K, cache):
    """Freed memory of the workspaces' sizes that holds anything but zeros."""
    for size in (K.kda_attn_workspace_size(cache), K.kda_kv_workspace_size(cache)):
        t = torch.full((size,), 0x5a, dtype=torch.uint8, device="cuda")
        del t
    torch.cuda.synchronize()


def fresh(K, seed):
    first, dense = make_cache(K, LENS, 2, 128, 64, BF, seed)
    dirty_blocks(K, first)
    cache = K.KdaKvCache(k=first.k, v=first.v, page_table=first.page_table, seq_lens=first.seq_lens, page_refs=first.page_refs)
    return cache, dense


def calls(K, cache, seed):
    """Queries, and the two attention calls over them into given outputs."""
    g = torch.Generator().manual_seed(seed)
    qd = torch.randn(4, 2, 8, 128, generator=g).to(BF)
    qp = torch.randn(90, 8, 128, generator=g).to(BF)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rows, one, cu, d, p = i32([0, 1, 2, 3]), i32([0]), i32([0, 90]), qd.cuda(), qp.cuda()
    out = torch.zeros_like(d), torch.zeros_like(p), torch.zeros(d.shape[:3], device="cuda"), torch.zeros(p.shape[:2], device="cuda")

    def run(**kw):
        K.kda_attn_decode(cache, 0, rows, d, out=out[0], lse=out[2], **kw)
        K.kda_attn_prefill(cache, 0, one, cu, 90, p, out=out[1], lse=out[3], **kw)

    def check(dense):
        assert K.kda_kv_get_error(cache) == 0
        for b, n in enumerate(LENS):
            check_attention(out[0][b], out[2][b], attention(qd[b].to(F64), *dense[b], n, 128 ** -0.5, 0, 0), BF, n)
        check_attention(out[1], out[3], attention(qp.to(F64), *dense[0], LENS[0], 128 ** -0.5, 0, 0), BF, LENS[0])
        for t in out:
            t.zero_()

    return run, check


@pytest.mark.gpu
def test_first_call_on_another_stream(K):
    """Work queued on the current stream does not come between the clear and a first call elsewhere."""
    cache, dense = fresh(K, 61)
    run, check = calls(K, cache, 62)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        a = a @ a * 1e-3   # the current stream is busy
    run(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    check(dense)


@pytest.mark.gpu
def test_a_capture_as_the_first_call(K):
    """Captured first, then called eagerly before any replay, then replayed, then called again."""
    cache, dense = fresh(K, 63)
    run, check = calls(K, cache, 64)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    run()
    check(dense)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        check(dense)
    run()
    check(dense)
    assert not cache.__dict__["_attn_ws"][:16384].any()   # the counters are ready for the next call


@pytest.mark.gpu
def test_a_cache_made_inside_a_capture_asks_for_a_workspace(K):
    cache, _ = fresh(K, 65)
    rows = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 1, 8, 128, dtype=BF, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        inner = K.KdaKvCache(k=cache.k, v=cache.v, page_table=cache.page_table, seq_lens=cache.seq_lens,
                             page_refs=cache.page_refs, err_word=cache.err_word)
        with pytest.raises(RuntimeError, match="captur"):
            K.kda_attn_decode(inner, 0, rows, q)
        q.zero_()   # (a graph with a node)
    torch.cuda.synchronize()
