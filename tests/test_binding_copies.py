"""Layers, pools, caches and rotations are copied and pickled after calls as before them: what was built of their tensors
(structs with addresses, plans, workspaces) stays behind and is built anew."""
from __future__ import annotations

import copy
import io
import pickle

import pytest
import torch

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def made(K, what, device="cpu"):
    if what == "rope":
        return K.KdaRope.make(32, scaling="yarn", factor=4.0, interleaved=True, device=device)
    if what == "cache":
        return K.KdaKvCache.zeros(1, 4, 2, 3, 2, 16, 64, dtype=torch.uint8, device=device)
    if what == "pool":
        return K.KdaPool.zeros(3, 2, device=device)
    z = lambda *s, dtype=F32: torch.zeros(s, dtype=dtype, device=device)
    return K.KdaLayer(z(256, 128, dtype=BF), z(2), z(256), z(3, 256, 4, dtype=BF), z(128))


def tensors(x):
    return {k: v for k, v in vars(x).items() if isinstance(v, torch.Tensor) and not k.startswith("_")}


def unpickled(x):
    f = io.BytesIO()
    torch.save(x, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


WAYS = [copy.deepcopy, copy.copy, lambda x: pickle.loads(pickle.dumps(x)), unpickled]


@pytest.mark.parametrize("way", WAYS, ids=["deepcopy", "copy", "pickle", "save"])
@pytest.mark.parametrize("what", ["rope", "cache", "pool", "layer"])
def test_after_a_call(K, what, way):
    x = made(K, what)
    x.c_struct()   # as a call does
    if what == "rope":
        pos, q = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 2, 64, dtype=BF)
        with pytest.raises(TypeError):   # (after its plan is made)
            K.kda_rope(x, pos, q)
        assert vars(x)["_plans"]
    y = way(x)
    assert type(y) is type(x) and tensors(y).keys() == tensors(x).keys()
    for k, t in tensors(x).items():
        u = tensors(y)[k]
        assert torch.equal(u.view(torch.uint8), t.view(torch.uint8)) and (u.data_ptr() == t.data_ptr()) == (way is copy.copy)
    for k, v in vars(x).items():
        if not k.startswith("_") and not isinstance(v, torch.Tensor):
            assert getattr(y, k) == v
    a, b = x.c_struct(), y.c_struct()
    assert a is not b
    for name, _ in a._fields_:
        u, v = getattr(a, name), getattr(b, name)
        assert u == v or way is not copy.copy and v in [t.data_ptr() for t in tensors(y).values()], name
    if what == "cache":
        for kind in ("_kv_ws", "_attn_ws"):
            assert vars(x)[kind].data_ptr() != vars(y)[kind].data_ptr() and not vars(y)[kind].any()


@pytest.mark.gpu
def test_a_copied_model_computes_the_same(K):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rope, cache = made(K, "rope", "cuda"), made(K, "cache", "cuda")
    x = torch.randn(2, 9, 8, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(BF)

    def step(rope, cache, x):
        rows = i32([2, 0])
        K.kda_kv_extend(cache, rows, x.shape[1])
        q = K.kda_kv_append_rope(cache, 0, rows, rope, x[:, :, :4], x[:, :, 4:6], x[:, :, 6:])
        return q, K.kda_attn_decode(cache, 0, rows, q)

    step(rope, cache, x[:, :8])
    held = cache.k.clone()
    r2, c2 = copy.deepcopy((rope, cache))
    r3, c3 = pickle.loads(pickle.dumps((rope, cache)))
    a = step(rope, cache, x[:, 8:])
    assert torch.equal(c2.k, held) and torch.equal(c3.k, held)   # copies have pages of their own
    for b, c in ((step(r2, c2, x[:, 8:]), c2), (step(r3, c3, x[:, 8:]), c3)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(c.k, cache.k)
        assert K.kda_kv_get_error(c) == 0
