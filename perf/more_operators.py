"""Rotary positions, appends that rotate on the way, and attention over a 4-bit cache: what is measured, and their plain forms.

The rotation turns pairs of a head's first ``rot`` elements by position * frequency; caches are pages ``k`` and ``v``
[layers, pages, Hkv, page size, D], a page table [rows, pages per row] (-1: no page) and lengths [rows].  A 4-bit cache
holds, for each page and head, the E2M1 codes of all its tokens (two elements a byte, the first in the low bits) and
then an E4M3 scale for each 16 elements: an element stands for layer scale * block scale * code.  ``run`` computes all
of it with elementary torch operations, or with ``own`` set through the package's entry points.
"""
import math
import random

import torch

own = False

NEG = float("-inf")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # of E2M1, the sign in the fourth bit


# ---------------------------------------------------------------- cases

def _rope(name, B, T, Hq, Hkv, D=128, rot=0, pairs="half", scaling="none", ctx=0, dtype="bf16", ragged=False):
    """Queries and keys of B sequences of T tokens (the longest, where ragged) behind contexts of up to ctx tokens."""
    c = dict(op="rope", B=B, q_len=T, ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, rot=rot or D, pairs=pairs, scaling=scaling, dtype=dtype,
             ragged=ragged)
    return dict(c, name=name) if name else c


def _append(name, B, T, ctx, Hq, Hkv, D=128, rot=0, pairs="half", scaling="none", ps=64, dtype="bf16", kv="same", ragged=False):
    c = dict(op="append", B=B, q_len=T, ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, rot=rot or D, pairs=pairs, scaling=scaling, ps=ps,
             dtype=dtype, kv=kv, ragged=ragged)
    return dict(c, name=name) if name else c


def _attn(name, op, B, q_len, ctx, Hq, Hkv, D=128, ps=64, dtype="bf16", window=0, sinks=0, ragged=False, rot=0, pairs="half"):
    """Attention over a 4-bit cache; "step": the new tokens are rotated and appended first."""
    c = dict(op=op, B=B, q_len=q_len, ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, ps=ps, dtype=dtype, kv="e2m1", window=window, sinks=sinks,
             ragged=ragged, rot=rot or D, pairs=pairs, scaling="none")
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token: nothing but latency
        _rope("rope_b1", 1, 1, 32, 8, ctx=517),
        # the prefill workload of the KDA layers, 4 x 4096, in the attention layer next to them, frequencies scaled by parts
        _rope("rope_b4_4096", 4, 4096, 32, 8, scaling="yarn"),
        # prompts of odd lengths far into long documents, adjacent pairs in half of a small head, fp16
        _rope("rope_part_odd", 5, 1999, 40, 8, D=64, rot=32, pairs="adjacent", scaling="linear", ctx=131072, dtype="fp16", ragged=True),
        # queries, keys and values of one decode step
        _append("append_rope_b64", 64, 1, 4096, 32, 8, ragged=True),
        # those of a prefill of 16 prompts, into an 8-bit cache
        _append("append_rope_prefill_e4m3", 16, 4096, 0, 32, 8, ps=32, kv="e4m3", ragged=True),
        # a layer's part of a decode step on a 4-bit cache: rotate, append, attend
        _attn("step_b64_e2m1", "step", 64, 1, 8192, 32, 8, ragged=True),
        # one user, a short chat
        _attn("decode_b1_e2m1", "decode", 1, 1, 517, 32, 8),
        # a large batch, the reason for a 4-bit cache
        _attn("decode_b256_e2m1", "decode", 256, 1, 4096, 32, 8, ps=32, ragged=True),
        # four draft tokens to verify in a sliding-window layer, an odd group of small heads, fp16
        _attn("verify_b64_t4_e2m1", "decode", 64, 4, 16384, 40, 8, D=64, ps=16, dtype="fp16", window=1024, sinks=4, ragged=True),
        # one long document read by one user: the cache's length has to be split
        _attn("decode_b1_long_e2m1", "decode", 1, 1, 131072, 64, 8, ps=128),
        # short prompts of odd lengths behind a shared context, one key head per query head
        _attn("prefill_odd_e2m1", "prefill", 5, 197, 131, 8, 8, D=64, ps=16, ragged=True),
        # 4 x 4096 tokens whose keys and values went to the 4-bit cache
        _attn("prefill_b4_4096_e2m1", "prefill", 4, 4096, 0, 32, 8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "step", "decode", "decode", "prefill"])
    D, ps = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 5, 8])
    rot = rng.choice([D, D, D // 2, D // 4])
    pairs, scaling = rng.choice(["half", "half", "adjacent"]), rng.choice(["none", "none", "linear", "yarn"])
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    sinks = rng.choice([0, 4, 19]) if window else 0
    ragged = rng.random() < 0.7
    if op == "rope":
        B = _log(rng, 1, 256)
        return _rope(None, B, _log(rng, 1, max(1, 16384 // B)), G * Hkv, Hkv, D, rot, pairs, scaling, rng.choice([0, _log(rng, 1, 1 << 20)]), dtype, ragged)
    if op == "append":
        B = _log(rng, 1, 256)
        return _append(None, B, _log(rng, 1, max(1, 32768 // B)), _log(rng, 1, 2048), min(G, 4) * Hkv, Hkv, D, rot, pairs, scaling, ps, dtype,
                       rng.choice(["same", "e4m3"]), ragged)
    if op == "prefill":
        B = _log(rng, 1, 16)
        return _attn(None, op, B, _log(rng, 17, 4096 // B + 17), rng.choice([0, _log(rng, 1, 4096)]), min(G, 4) * Hkv, Hkv, D, ps, dtype, window, sinks, ragged)
    B = _log(rng, 1, 256)
    ctx = _log(rng, 1, max(16, min(65536, 262144 // B)))
    T = rng.choice([1, 1, 2, 5, 16])
    if op == "step":
        return _attn(None, op, B, T, ctx, G * Hkv, Hkv, D, ps, dtype, window, sinks, ragged, rot if pairs == "adjacent" else max(rot, 32), pairs)
    return _attn(None, op, B, T, ctx, G * Hkv, Hkv, D, ps, dtype, window, sinks, ragged)


# ---------------------------------------------------------------- inputs

def _spread(n, most, ragged, salt):
    """n lengths: all `most`, or spread over the logarithm of 1..most with the longest among them."""
    if not ragged:
        return [most] * n
    r = random.Random(salt * 1000003 + n * 8191 + most)
    got = [min(most, max(1, int(math.exp(r.uniform(0.0, math.log(most + 1)))))) for _ in range(n)]
    for i in range(0, n, 2):   # and every other one over the upper half
        got[i] = r.randint(max(1, most // 2), most)
    got[r.randrange(n)] = most
    return got


def _lengths(case):
    """(new tokens, all tokens) of each sequence."""
    B, q_len, ctx = case["B"], case["q_len"], case["ctx"]
    if case["op"] in ("decode", "step"):
        total = [max(q_len, x) for x in _spread(B, ctx, case["ragged"], 1)]
        return [q_len] * B, total
    new = _spread(B, q_len, case["ragged"], 2)
    old = _spread(B, ctx, case["ragged"], 3) if ctx else [0] * B
    return new, [a + b for a, b in zip(new, old)]


def _seen(new, total, window, sinks):
    """Visible (query, key) pairs of a sequence's new tokens, and the keys that at least one of them sees."""
    pairs, first = 0, total - new
    for p in range(first, total) if window else ():
        lo = max(0, p - window + 1)
        pairs += p + 1 - lo + min(sinks, lo)
    if not window:
        return new * first + new * (new + 1) // 2, total
    lo = max(0, first - window + 1)
    return pairs, total - lo + min(sinks, lo)


def _frequencies(case):
    """(radians per position of each pair, what cosines and sines are multiplied with)."""
    rot, base, factor, length = case["rot"], 10000.0, 8.0, 4096
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if case["scaling"] == "yarn":   # slow pairs are slowed down, fast ones kept, a ramp between the two
        at = lambda turns: rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(32.0))), min(rot - 1, math.ceil(at(1.0)))
        keep = [1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        return [x * k + x / factor * (1.0 - k) for x, k in zip(f, keep)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _e2m1(y):
    """Codes of y, to the nearest, ties to the even code, 6 at most."""
    a = y.abs()
    code = (a > 0.25).to(torch.uint8)
    for t, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= t) if up else (a > t)
    return code | torch.signbit(y).to(torch.uint8) << 3


def _blocks(x, scale):
    """x [..., D] -> (packed codes [..., D / 2], E4M3 scales [..., D / 16]); `scale`: the layer's, to be divided by first."""
    y = (x / scale).unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1) / 6.0).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    c = _e2m1(y / s.to(y.dtype)[..., None]).flatten(-2)
    return c[..., 0::2] | c[..., 1::2] << 4, s


def _fill(shape, kv, scale, gen):
    """A random cache of this shape: values around one."""
    layers, pages, Hkv, ps, D = shape
    if kv == "e2m1":
        out = torch.empty(layers, pages, Hkv, ps * (D // 2 + D // 16), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (Hkv * ps * D))
        for layer in range(layers):
            for a in range(0, pages, step):
                n = min(step, pages - a)
                x = torch.randn(n, Hkv, ps, D, device="cuda", generator=gen)
                c, s = _blocks(x, scale[layer][None, :, None, None])
                out[layer, a:a + n] = torch.cat([c.flatten(-2), s.view(torch.uint8).flatten(-2)], -1)
        return out.view(layers, pages, Hkv, ps, D // 2 + D // 16)
    out = torch.empty(shape, dtype=TYPES[kv], device="cuda")
    for layer in range(layers):
        x = torch.randn(shape[1:], device="cuda", generator=gen, dtype=torch.float32)
        out[layer] = (x * 50).clamp_(-448, 448).to(out.dtype) if kv == "e4m3" else x.to(out.dtype)
    return out


def _tables(counts, width, pages, gen):
    """A page table whose rows take counts[r] pages each, in random order, and the count of users per page."""
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    start = torch.tensor([0] + counts, device="cuda").cumsum(0)[:-1, None]
    j = torch.arange(width, device="cuda")[None]
    held = j < torch.tensor(counts, device="cuda")[:, None]
    table = torch.where(held, order[(start + j).clamp_(max=pages - 1)], -1).to(torch.int32)
    refs = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    refs.index_add_(0, table.reshape(-1).long() % (pages + 1), torch.ones(table.numel(), dtype=torch.int32, device="cuda"))
    return table, refs[:pages].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    op, D, Hq, Hkv, B = case["op"], case["D"], case["Hq"], case["Hkv"], case["B"]
    dtype = TYPES[case["dtype"]]
    new, total = _lengths(case)
    s = dict(case=case, freqs=_frequencies(case))
    # the projections leave q, k and v side by side in one buffer
    qkv = torch.randn(sum(new), (Hq + 2 * Hkv) * D, device="cuda", generator=gen).to(dtype)
    s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    s["k_new"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    s["v_new"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    if op == "rope":
        s["pos"] = torch.cat([torch.arange(t - n, t, device="cuda", dtype=torch.int32) for n, t in zip(new, total)])
        return s
    ps, kv = case["ps"], case["dtype"] if case["kv"] == "same" else case["kv"]
    counts = [-(-x // ps) for x in total]
    pages, width = sum(counts) + 7, max(counts) + 1
    table, refs = _tables(counts, width, pages, gen)
    order = torch.randperm(B, device="cuda", generator=gen)   # sequences hold the cache's rows in any order
    place = torch.argsort(order)
    if kv in ("e4m3", "e2m1"):
        lo = 0.015 if kv == "e4m3" else 0.5
        s.update(k_scale=lo * (1 + torch.rand(1, Hkv, device="cuda", generator=gen)),
                 v_scale=lo * (1 + torch.rand(1, Hkv, device="cuda", generator=gen)))
    s.update(k=_fill((1, pages, Hkv, ps, D), kv, s.get("k_scale"), gen), v=_fill((1, pages, Hkv, ps, D), kv, s.get("v_scale"), gen),
             table=table[place].contiguous(), refs=refs, rows=order.to(torch.int32),
             lens=_ints(total)[place].contiguous(), max_len=max(new), total=sum(new), cu=_ints([0] + new).cumsum(0).to(torch.int32))
    if op in ("decode", "step"):
        for name in ("q", "k_new", "v_new"):
            s[name] = s[name].unflatten(0, (B, case["q_len"]))
    s["even"] = all(x == new[0] for x in new)
    return s


# ---------------------------------------------------------------- plain forms

def _rotated(x, pos, case, freqs):
    """x [N, H, D] turned to positions pos [N], in 32 bits (the angles in 64)."""
    f, m = freqs
    a = pos.double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
    cos, sin = (torch.cos(a) * m).float()[:, None], (torch.sin(a) * m).float()[:, None]
    x, rot = x.float(), case["rot"]
    if case["pairs"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _places(s):
    """Of every new token: page, place in the page and position."""
    c, rows, cu = s["case"], s["rows"].long(), s["cu"].long()
    tok = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu, tok, right=True) - 1
    pos = s["lens"][rows[b]].long() - (cu[b + 1] - cu[b]) + tok - cu[b]
    return s["table"][rows[b], pos // c["ps"]].long(), pos % c["ps"], pos


def _plain_append(s):
    """Rotated queries, after the rotated keys and the values went to their pages."""
    c = s["case"]
    flat = lambda x: x.flatten(0, 1) if x.dim() == 4 else x  # noqa: E731
    page, at, pos = _places(s)
    for name, x in (("k", _rotated(flat(s["k_new"]), pos, c, s["freqs"])), ("v", flat(s["v_new"]).float())):
        cache = s[name][0]
        if c["kv"] == "e2m1":
            codes, scales = _blocks(x, s[name + "_scale"][0][None, :, None])
            D, ps = c["D"], c["ps"]
            raw = cache.flatten(-2)
            raw[:, :, :ps * D // 2].unflatten(-1, (ps, D // 2))[page, :, at] = codes
            raw[:, :, ps * D // 2:].unflatten(-1, (ps, D // 16))[page, :, at] = scales.view(torch.uint8)
        else:
            if c["kv"] == "e4m3":
                x = (x / s[name + "_scale"][0][None, :, None]).clamp(-448, 448)
            cache[page, :, at] = x.to(cache.dtype)
    return _rotated(flat(s["q"]), pos, c, s["freqs"]).to(s["q"].dtype).view(s["q"].shape)


def _pair_table():
    """The two values of each byte of codes."""
    v = torch.tensor(CODES + tuple(-x for x in CODES), device="cuda")
    b = torch.arange(256, device="cuda")
    return torch.stack([v[b & 15], v[b >> 4]], -1)


def _dense(pages, table, rows, scale, D):
    """[B, Hkv, tokens, D] in 32 bits of the sequences' pages in a 4-bit cache."""
    x = pages[table[rows.long()].clamp(min=0).long()]              # [B, width, Hkv, ps, bytes]
    ps = x.shape[3]
    x = x.flatten(-2)
    c = torch.index_select(_pair_table(), 0, x[..., :ps * D // 2].reshape(-1).int())
    c = c.view(*x.shape[:3], ps, D // 16, 16)
    c *= x[..., ps * D // 2:].view(torch.float8_e4m3fn).float().view(*x.shape[:3], ps, D // 16, 1)
    return c.flatten(-2).transpose(1, 2).flatten(2, 3) * scale[None, :, None, None]


def _plain_attention(s, q, n):
    """q [B, T, Hq, D] with n[b] tokens each -> out in 32 bits, log of the sum."""
    c = s["case"]
    B, T, Hq, D = q.shape
    Hkv, G = c["Hkv"], Hq // c["Hkv"]
    k = _dense(s["k"][0], s["table"], s["rows"], s["k_scale"][0], D)
    v = _dense(s["v"][0], s["table"], s["rows"], s["v_scale"][0], D)
    total = s["lens"][s["rows"].long()].long()
    j = torch.arange(k.shape[2], device=k.device)
    p = (total - n)[:, None] + torch.arange(T, device=k.device)      # [B, T]
    see = j <= p[..., None]
    if c["window"]:
        see &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    held = (j < total[:, None])[:, None, :, None]
    k, v = torch.where(held, k, 0.0), torch.where(held, v, 0.0)
    qg = q.float().unflatten(2, (Hkv, G)).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    a = qg @ k.transpose(2, 3)
    a *= 1.0 / math.sqrt(D)
    a = a.view(B, Hkv, T, G, -1).masked_fill_(~see[:, None, :, None], NEG)
    m = a.amax(-1, keepdim=True)
    a -= torch.where(m == NEG, 0.0, m)
    a.exp_()
    l = a.sum(-1, keepdim=True)
    o = (a.view(B, Hkv, T * G, -1) @ v).view(B, Hkv, T, G, D) / torch.where(l == 0, 1.0, l)
    lse = (m + torch.log(l)).squeeze(-1)
    return (o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(q.dtype),
            lse.permute(0, 2, 1, 3).reshape(B, T, Hq))


# ---------------------------------------------------------------- one pass

def _handles(s):
    """The package's rotation and its cache over this state's tensors, made once as a program keeps them."""
    if "K" not in s:
        import verify_kda_decode_gb300 as K
        c = s["case"]
        s["rope"] = K.KdaRope.from_frequencies(s["freqs"][0], interleaved=c["pairs"] == "adjacent", scale=s["freqs"][1])
        if c["op"] != "rope":
            s["cache"] = K.KdaKvCache(k=s["k"], v=s["v"], page_table=s["table"], seq_lens=s["lens"], page_refs=s["refs"],
                                      k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
        s["K"] = K
    return s["K"], s["rope"], s.get("cache")


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        K, rope, cache = _handles(s)
        if op == "rope":
            return K.kda_rope(rope, s["pos"], s["q"], s["k_new"])
        if op == "append":
            q = K.kda_kv_append_rope(cache, 0, s["rows"], rope, s["q"], s["k_new"], s["v_new"], cu_seqlens=None if s["even"] else s["cu"])
            return q, s["k"], s["v"]
        if op == "step":
            q = K.kda_kv_append_rope(cache, 0, s["rows"], rope, s["q"], s["k_new"], s["v_new"])
            out, lse = K.kda_attn_decode(cache, 0, s["rows"], q, window=c["window"], sinks=c["sinks"], return_lse=True)
            return q, out, lse
        if op == "decode":
            return K.kda_attn_decode(cache, 0, s["rows"], s["q"], window=c["window"], sinks=c["sinks"], return_lse=True)
        return K.kda_attn_prefill(cache, 0, s["rows"], s["cu"], s["max_len"], s["q"], window=c["window"], sinks=c["sinks"],
                                  return_lse=True)
    if op == "rope":
        return tuple(_rotated(x, s["pos"], c, s["freqs"]).to(x.dtype) for x in (s["q"], s["k_new"]))
    if op == "append":
        return _plain_append(s), s["k"], s["v"]
    if op == "step":
        q = _plain_append(s)
        return (q,) + _plain_attention(s, q, c["q_len"])
    if op == "decode":
        return _plain_attention(s, s["q"], c["q_len"])
    cu, T = s["cu"].long(), s["max_len"]
    n = cu[1:] - cu[:-1]
    t = torch.arange(T, device="cuda")
    valid = t < n[:, None]
    at = (cu[:-1, None] + t).clamp(max=s["total"] - 1)
    out, lse = _plain_attention(s, s["q"][at], n)
    return out[valid], lse[valid]


def work(case):
    D, Hq, Hkv, op = case["D"], case["Hq"], case["Hkv"], case["op"]
    new, total = _lengths(case)
    n = sum(new)
    turn = n * (Hq + Hkv) * case["rot"] * 3
    if op == "rope":
        return {"bytes": n * (Hq + Hkv) * D * 4 + n * 4, "flops": turn}
    key = D * 2 if case["kv"] == "same" else D if case["kv"] == "e4m3" else D // 2 + D // 16   # bytes of a key
    moved = n * (Hq * D * 4 + 2 * Hkv * (D * 2 + key))
    if op == "append":
        return {"bytes": moved, "flops": turn}
    seen = [_seen(a, b, case["window"], case["sinks"]) for a, b in zip(new, total)]
    bytes_ = sum(x[1] for x in seen) * Hkv * key * 2 + n * Hq * (D * 4 + 4)
    flops = sum(x[0] for x in seen) * Hq * D * 4
    return {"bytes": bytes_ + moved, "flops": flops + turn} if op == "step" else {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------- in 64 bits

def _turned(x, pos, case, freqs):
    """The rotation as products of complex numbers of 64 bits."""
    rot, (f, m) = case["rot"], freqs
    angle = torch.outer(pos.to(torch.float64), torch.tensor(f, dtype=torch.float64, device="cuda"))
    unit = torch.polar(torch.full_like(angle, m), angle)[:, None]
    x = x.to(torch.float64)
    head = x[..., :rot]
    if case["pairs"] == "half":
        z = torch.complex(*(t.contiguous() for t in head.chunk(2, -1))) * unit
        head = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * unit
        head = torch.view_as_real(z).flatten(-2)
    return torch.cat([head, x[..., rot:]], -1)


def _nearest(x, scale):
    """x [n, Hkv, D] as a 4-bit cache holds it, in 64 bits: nearest values by distance, of two the one with the even code."""
    grid = torch.tensor(CODES, dtype=torch.float64, device="cuda")
    y = (x / scale[:, None]).unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn).to(torch.float64)
    far = ((y / s).abs()[..., None] - grid).abs()
    far = far + torch.tensor([0.0, 1e-15] * 4, dtype=torch.float64, device="cuda")
    return (grid[far.argmin(-1)] * torch.sign(y) * s).flatten(-2) * scale[:, None]


def _stored(s, name, row, L, D):
    """A row's keys or values [L, Hkv, D] in a 4-bit cache, in 64 bits."""
    ps = s["case"]["ps"]
    raw = s[name][0, s["table"][row, :-(-L // ps)].long()].flatten(-2)      # [pages, Hkv, bytes]
    byte = raw[..., :ps * D // 2].unflatten(-1, (ps, D // 2))
    nib = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).long()
    mag = torch.tensor(CODES, dtype=torch.float64, device="cuda")[nib & 7] * (1.0 - 2.0 * (nib >> 3).double())
    sc = raw[..., ps * D // 2:].contiguous().view(torch.float8_e4m3fn).double().unflatten(-1, (ps, D // 16))
    x = mag * sc.repeat_interleave(16, -1) * s[name + "_scale"][0].double()[:, None, None]
    return x.transpose(1, 2).flatten(0, 1)[:L]


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, sequence by sequence."""
    s = prepare(case, seed)
    new, total = _lengths(case)
    D, Hkv, Hq, op = case["D"], case["Hkv"], case["Hq"], case["op"]
    f64 = torch.float64
    if op == "rope":
        return tuple(_turned(x, s["pos"], case, s["freqs"]) for x in (s["q"], s["k_new"]))
    flat = {name: s[name].flatten(0, 1) if s[name].dim() == 4 else s[name] for name in ("q", "k_new", "v_new")}
    if op in ("append", "step"):
        pos = torch.cat([torch.arange(t - n, t, device="cuda") for n, t in zip(new, total)])
        q, k_new, v_new = _turned(flat["q"], pos, case, s["freqs"]), _turned(flat["k_new"], pos, case, s["freqs"]), flat["v_new"].to(f64)
    if op == "append":
        k, v, at = s["k"].to(f64), s["v"].to(f64), 0
        for b, n in enumerate(new):
            row = int(s["rows"][b])
            p = torch.arange(total[b] - n, total[b], device="cuda")
            page = s["table"][row].long()[p // case["ps"]]
            for cache, x, sc in ((k, k_new, s.get("k_scale")), (v, v_new, s.get("v_scale"))):
                y = x[at:at + n]
                if sc is not None:
                    y = (y / sc[0].to(f64)[:, None]).clamp(-448.0, 448.0)
                cache[0, page, :, p % case["ps"]] = y
            at += n
        return q, k, v
    turned = q if op == "step" else None
    q = (q.to(flat["q"].dtype) if op == "step" else flat["q"]).to(f64)   # attention takes the queries in their type
    G = Hq // Hkv
    out = torch.zeros(q.shape, dtype=f64, device="cuda")
    lse = torch.full(q.shape[:2], NEG, dtype=f64, device="cuda")
    at = 0
    for b, n in enumerate(new):
        row, L = int(s["rows"][b]), total[b]
        k, v = _stored(s, "k", row, L, D), _stored(s, "v", row, L, D)
        if op == "step":   # the new tokens as the cache holds them
            k[L - n:] = _nearest(k_new[at:at + n], s["k_scale"][0].to(f64))
            v[L - n:] = _nearest(v_new[at:at + n], s["v_scale"][0].to(f64))
        i, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
        hidden = j > i
        if case["window"]:
            hidden |= (j <= i - case["window"]) & (j >= case["sinks"])
        for h in range(Hq):
            w = ((q[at:at + n, h] @ k[:, h // G].T) / D ** 0.5).masked_fill(hidden, NEG)
            lse[at:at + n, h] = torch.logsumexp(w, 1)
            out[at:at + n, h] = torch.softmax(w, 1) @ v[:, h // G]
        at += n
    shape = s["q"].shape
    got = out.view(shape), lse.view(shape[:-1])
    return (turned.view(shape),) + got if op == "step" else got
