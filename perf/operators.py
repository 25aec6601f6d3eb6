"""The attention layers' operators over a paged key-value cache: what is measured, and their plain forms.

Every operator works on a cache of pages: ``k`` and ``v`` [layers, pages, Hkv, page size, D], a page table
[rows, pages per row] (-1: no page), lengths [rows] and a count of users per page.  ``run`` computes them with
elementary torch operations, or with ``own`` set through the package's entry points.
"""
import math
import random

import torch

own = False

NEG = float("-inf")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------- cases

def _attn(name, op, B, q_len, ctx, Hq, Hkv, D=128, ps=64, dtype="bf16", kv="same", window=0, sinks=0, ragged=False):
    """B sequences of q_len new tokens on top of a context of ctx tokens (q_len and ctx are the longest ones where ragged)."""
    c = dict(op=op, B=B, q_len=q_len, ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, ps=ps, dtype=dtype, kv=kv, window=window,
             sinks=sinks, ragged=ragged)
    return dict(c, name=name) if name else c


def _append(name, B, q_len, ctx, Hkv, D=128, ps=64, dtype="bf16", kv="same", ragged=False):
    c = dict(op="append", B=B, q_len=q_len, ctx=ctx, Hkv=Hkv, D=D, ps=ps, dtype=dtype, kv=kv, ragged=ragged)
    return dict(c, name=name) if name else c


def _pages(name, op, rows, fan, ctx, layers, pages, Hkv, D=128, ps=64, kv="bf16", drafts=4):
    """rows sequences of up to ctx tokens; fan copies of each (fork), or a share of them gone (compact: one of fan)."""
    c = dict(op=op, rows=rows, fan=fan, ctx=ctx, layers=layers, pages=pages, Hkv=Hkv, D=D, ps=ps, kv=kv, drafts=drafts)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, a short chat: nothing but latency
        _attn("decode_b1", "decode", 1, 1, 517, 32, 8),
        # a full decode step of a server, lengths from one token to 8192
        _attn("decode_b64_ragged", "decode", 64, 1, 8192, 32, 8, ragged=True),
        # a large batch on an 8-bit cache
        _attn("decode_b256_e4m3", "decode", 256, 1, 4096, 32, 8, ps=32, kv="e4m3", ragged=True),
        # four draft tokens to verify in a sliding-window layer, an odd group of heads, small heads, fp16
        _attn("verify_b64_t4_window", "decode", 64, 4, 16384, 40, 8, D=64, ps=16, dtype="fp16", window=1024, sinks=4,
              ragged=True),
        # one long document read by one user: the cache's length has to be split
        _attn("decode_b1_long", "decode", 1, 1, 131072, 64, 8, ps=128),
        # short prompts of odd lengths behind a shared context, one key head per query head
        _attn("prefill_odd", "prefill", 5, 197, 131, 8, 8, D=64, ps=16, ragged=True),
        # the prefill workload of the KDA layers, 4 x 4096, in the full-attention layer next to them
        _attn("prefill_b4_4096", "prefill", 4, 4096, 0, 32, 8),
        # a long prompt in a sliding-window layer
        _attn("prefill_window_16k", "prefill", 1, 16384, 0, 8, 2, window=2048, sinks=4),
        # the keys and values of one decode step
        _append("append_b64", 64, 1, 4096, 8),
        # those of a prefill of 16 prompts into an 8-bit cache
        _append("append_prefill_e4m3", 16, 4096, 0, 8, ps=32, kv="e4m3", ragged=True),
        # parallel sampling: prompts forked, drafts reserved and most of them given back
        _pages("fork_b64", "fork", 16, 4, 8192, 4, 4096, 4),
        # a fragmented cache closed up
        _pages("compact_4k_pages", "compact", 64, 2, 4096, 4, 4096, 4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "fork", "compact"])
    D, ps = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    dtype, kv = rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["same", "same", "e4m3"])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 5, 8])
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    sinks = rng.choice([0, 4, 19]) if window else 0
    if op == "decode":
        B = _log(rng, 1, 256)
        ctx = _log(rng, 1, max(16, min(65536, 262144 // B)))
        return _attn(None, op, B, rng.choice([1, 1, 2, 5, 16]), ctx, G * Hkv, Hkv, D, ps, dtype, kv, window, sinks,
                     rng.random() < 0.7)
    if op == "prefill":
        B = _log(rng, 1, 16)
        q_len = _log(rng, 17, 4096 // B + 17)
        G = min(G, 4)
        return _attn(None, op, B, q_len, rng.choice([0, _log(rng, 1, 4096)]), G * Hkv, Hkv, D, ps, dtype, kv, window,
                     sinks, rng.random() < 0.7)
    if op == "append":
        B = _log(rng, 1, 256)
        return _append(None, B, _log(rng, 1, max(1, 65536 // B // 2)), _log(rng, 1, 2048), Hkv, D, ps, dtype, kv,
                       rng.random() < 0.7)
    ps = rng.choice([32, 64, 128])
    rows, fan = _log(rng, 2, 64), rng.choice([2, 3, 4])
    ctx = _log(rng, ps, 65536 // rows)
    pages = rows * (ctx // ps + 1) + rows * fan * 3 + rng.randrange(200)
    return _pages(None, op, rows, fan, ctx, rng.choice([1, 2, 4]), pages, rng.choice([1, 2, 4]), D, ps,
                  rng.choice(["bf16", "e4m3"]), rng.choice([1, 4, 7]))


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
    if case["op"] == "decode":
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


def _fill(shape, dtype, gen):
    """A random cache of this shape: values around one, in codes of an 8-bit cache around 50."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for layer in range(shape[0]):
        x = torch.randn(shape[1:], device="cuda", generator=gen, dtype=torch.float32)
        out[layer] = (x * 50).clamp_(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)
    return out


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


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
    op, ps, D, Hkv = case["op"], case["ps"], case["D"], case["Hkv"]
    s = dict(case=case)
    if op in ("fork", "compact"):
        kv = TYPES[case["kv"]]
        n = case["rows"]
        r = random.Random(int(seed))
        lens = [max(1, case["ctx"] - r.randrange(case["ctx"] // 4 + 1)) for _ in range(n)]
        width = -(-(case["ctx"] + case["drafts"]) // ps) + 1
        rows = n * (1 + case["fan"]) if op == "fork" else n
        counts = [-(-x // ps) for x in lens] + [0] * (rows - n)
        while sum(counts) + n * case["fan"] * 2 > case["pages"]:   # a cache too small for the longest prompts
            i = counts.index(max(counts))
            counts[i] -= 1
            lens[i] = counts[i] * ps - 1
        if op == "compact":   # some of the sequences have gone
            counts = [0 if i % case["fan"] else x for i, x in enumerate(counts)]
            lens = [0 if i % case["fan"] else x for i, x in enumerate(lens)]
        table, refs = _tables(counts, width, case["pages"], gen)
        s.update(k=_fill((case["layers"], case["pages"], Hkv, ps, D), kv, gen),
                 v=_fill((case["layers"], case["pages"], Hkv, ps, D), kv, gen), table=table, refs=refs,
                 lens=_ints(lens + [0] * (rows - n)))
        if op == "fork":
            s.update(src=_ints([i % n for i in range(n * case["fan"])]), dst=_ints(list(range(n, rows))),
                     drafts=_ints([case["drafts"]] * (n * case["fan"])),
                     keep=_ints([lens[i % n] + r.randint(0, case["drafts"]) for i in range(n * case["fan"])]))
        else:
            s.update(table0=table.clone(), refs0=refs.clone())
        if kv == torch.float8_e4m3fn:
            s.update(k_scale=torch.full((case["layers"], Hkv), 0.02, device="cuda"),
                     v_scale=torch.full((case["layers"], Hkv), 0.02, device="cuda"))
        return s
    dtype = TYPES[case["dtype"]]
    kv = dtype if case["kv"] == "same" else TYPES[case["kv"]]
    B = case["B"]
    new, total = _lengths(case)
    counts = [-(-x // ps) for x in total]
    pages, width = sum(counts) + 7, max(counts) + 1
    table, refs = _tables(counts, width, pages, gen)
    order = torch.randperm(B, device="cuda", generator=gen)   # sequences hold the cache's rows in any order
    place = torch.argsort(order)
    s.update(k=_fill((1, pages, Hkv, ps, D), kv, gen), v=_fill((1, pages, Hkv, ps, D), kv, gen),
             table=table[place].contiguous(), refs=refs, rows=order.to(torch.int32),
             lens=_ints(total)[place].contiguous(), max_len=max(new), total=sum(new))
    if kv == torch.float8_e4m3fn:
        s.update(k_scale=(0.015 + 0.01 * torch.rand(1, Hkv, device="cuda", generator=gen)),
                 v_scale=(0.015 + 0.01 * torch.rand(1, Hkv, device="cuda", generator=gen)))
    # the projections leave q, k and v side by side in one buffer
    Hq = case.get("Hq", 0)
    qkv = torch.randn(sum(new), (Hq + 2 * Hkv) * D, device="cuda", generator=gen).to(dtype)
    s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D)) if Hq else None
    s["k_new"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    s["v_new"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    s["cu"] = _ints([0] + new).cumsum(0).to(torch.int32)
    if op == "decode":
        s["q"] = s["q"].unflatten(0, (B, case["q_len"]))
    if op == "append" and all(x == new[0] for x in new):
        s["even"] = new[0]
    return s


# ---------------------------------------------------------------- plain forms

def _dense(pages, table, rows, scale):
    """[B, Hkv, tokens, D] in 32 bits of the sequences' pages."""
    x = pages[table[rows.long()].clamp(min=0).long()].float()        # [B, width, Hkv, ps, D]
    x = x.transpose(1, 2).flatten(2, 3)
    return x if scale is None else x * scale[None, :, None, None]


def _plain_attention(s, q, n):
    """q [B, T, Hq, D] with n[b] tokens each -> out in 32 bits, log of the sum."""
    c = s["case"]
    B, T, Hq, D = q.shape
    Hkv, G = c["Hkv"], Hq // c["Hkv"]
    ks, vs = s.get("k_scale"), s.get("v_scale")
    k = _dense(s["k"][0], s["table"], s["rows"], None if ks is None else ks[0])
    v = _dense(s["v"][0], s["table"], s["rows"], None if vs is None else vs[0])
    total = s["lens"][s["rows"].long()].long()
    j = torch.arange(k.shape[2], device=k.device)
    p = (total - n)[:, None] + torch.arange(T, device=k.device)      # [B, T]
    see = j <= p[..., None]
    if c["window"]:
        see &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    v = torch.where((j < total[:, None])[:, None, :, None], v, 0.0)
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


def _plain_append(s):
    c, rows = s["case"], s["rows"].long()
    cu = s["cu"].long()
    tok = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu, tok, right=True) - 1
    pos = s["lens"][rows[b]].long() - (cu[b + 1] - cu[b]) + tok - cu[b]
    page = s["table"][rows[b], pos // c["ps"]].long()
    at = pos % c["ps"]
    for name in ("k", "v"):
        x = s[name + "_new"].float()
        if c["kv"] == "e4m3":
            x = (x / s[name + "_scale"][0][None, :, None]).clamp(-448, 448)
        s[name][0][page, :, at] = x.to(s[name].dtype)


def _plain_fork(s):
    c, P, ps = s["case"], s["refs"].numel(), s["case"]["ps"]
    table, refs, lens, src, dst = s["table"], s["refs"], s["lens"], s["src"].long(), s["dst"].long()
    # the copies' old pages are dropped, then they share the pages of their sources
    old, new = table[dst], table[src]
    refs.index_add_(0, old[old >= 0].long(), -torch.ones_like(old[old >= 0]))
    refs.index_add_(0, new[new >= 0].long(), torch.ones_like(new[new >= 0]))
    table[dst] = new
    lens[dst] = lens[src]
    # room for the drafts: the lowest free pages, and a copy of a last page that others use too
    at, n = lens[dst].long(), s["drafts"].long()
    have = (at + ps - 1) // ps
    need = (at + n + ps - 1) // ps - have
    tail = table[dst, (have - 1).clamp(min=0)].long()
    copy = (at % ps != 0) & (n > 0) & (refs[tail.clamp(min=0)] > 1)
    want = need + copy
    off = want.cumsum(0) - want
    free = torch.nonzero(refs == 0).squeeze(1)
    j = torch.arange(table.shape[1], device="cuda")[None]
    added = (j >= have[:, None]) & (j < (have + need)[:, None])
    row = table[dst]
    pick = (off + copy)[:, None] + j - have[:, None]
    row = torch.where(added, free[pick.clamp(0, len(free) - 1)].to(torch.int32), row)
    fresh = free[off.clamp(max=len(free) - 1)]
    row = torch.where(copy[:, None] & (j == (have - 1)[:, None]), fresh[:, None].to(torch.int32), row)
    table[dst] = row
    refs[row[added].long()] = 1
    refs.index_add_(0, tail[copy], -torch.ones_like(tail[copy], dtype=torch.int32))
    refs[fresh[copy]] = 1
    filled = (torch.arange(ps, device="cuda")[None] < (at % ps)[copy][:, None])[None, :, None, :, None]
    for x in (s["k"], s["v"]):
        raw = x.view(torch.uint8) if c["kv"] == "e4m3" else x
        raw[:, fresh[copy]] = torch.where(filled, raw[:, tail[copy]], raw[:, fresh[copy]])
    lens[dst] = (at + n).to(torch.int32)
    # and the drafts that were not accepted given back
    keep = s["keep"].long()
    row = table[dst]
    gone = (j >= ((keep + ps - 1) // ps)[:, None]) & (row >= 0)
    refs.index_add_(0, row[gone].long(), -torch.ones_like(row[gone]))
    table[dst] = torch.where(gone, -1, row)
    lens[dst] = keep.to(torch.int32)


def _plain_compact(s):
    table, refs, P = s["table"], s["refs"], s["refs"].numel()
    live = refs > 0
    n = live.sum()
    ids = torch.arange(P, device="cuda")
    high = torch.nonzero(live & (ids >= n)).squeeze(1)
    low = torch.nonzero(~live & (ids < n)).squeeze(1)
    remap = torch.where(live, ids, -1)
    remap[high] = low
    for x in (s["k"], s["v"]):
        raw = x.view(torch.uint8) if s["case"]["kv"] == "e4m3" else x
        raw[:, low] = raw[:, high]
    refs[low] = refs[high]
    refs[high] = 0
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()].to(torch.int32), -1))
    return remap.to(torch.int32)


# ---------------------------------------------------------------- one pass

def _cache(s):
    """The package's cache over this state's tensors, made once as a program keeps it."""
    if "cache" not in s:
        import verify_kda_decode_gb300 as K
        s["cache"] = K.KdaKvCache(k=s["k"], v=s["v"], page_table=s["table"], seq_lens=s["lens"], page_refs=s["refs"],
                                  k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
        s["K"] = K
    return s["K"], s["cache"]


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        K, cache = _cache(s)
        if op == "decode":
            return K.kda_attn_decode(cache, 0, s["rows"], s["q"], window=c["window"], sinks=c["sinks"], return_lse=True)
        if op == "prefill":
            return K.kda_attn_prefill(cache, 0, s["rows"], s["cu"], s["max_len"], s["q"], window=c["window"],
                                      sinks=c["sinks"], return_lse=True)
        if op == "append":
            if "even" in s:
                K.kda_kv_append(cache, 0, s["rows"], s["k_new"], s["v_new"])
            else:
                K.kda_kv_append(cache, 0, s["rows"], s["k_new"], s["v_new"], cu_seqlens=s["cu"])
            return s["k"], s["v"]
        if op == "fork":
            K.kda_kv_fork(cache, s["src"], s["dst"])
            K.kda_kv_extend(cache, s["dst"], s["drafts"])
            K.kda_kv_truncate(cache, s["dst"], s["keep"])
            return s["k"], s["v"], s["table"], s["refs"], s["lens"]
        s["table"].copy_(s["table0"])   # fragmented again
        s["refs"].copy_(s["refs0"])
        remap = K.kda_kv_compact(cache)
        return s["k"], s["v"], s["table"], s["refs"], remap
    if op == "decode":
        return _plain_attention(s, s["q"], c["q_len"])
    if op == "prefill":
        cu, T = s["cu"].long(), s["max_len"]
        n = cu[1:] - cu[:-1]
        t = torch.arange(T, device="cuda")
        valid = t < n[:, None]
        at = (cu[:-1, None] + t).clamp(max=s["total"] - 1)
        out, lse = _plain_attention(s, s["q"][at], n)
        return out[valid], lse[valid]
    if op == "append":
        _plain_append(s)
        return s["k"], s["v"]
    if op == "fork":
        _plain_fork(s)
        return s["k"], s["v"], s["table"], s["refs"], s["lens"]
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    remap = _plain_compact(s)
    return s["k"], s["v"], s["table"], s["refs"], remap


def work(case):
    ps, D, Hkv = case["ps"], case["D"], case["Hkv"]
    if case["op"] in ("fork", "compact"):
        page = 2 * case["layers"] * Hkv * ps * D * (1 if case["kv"] == "e4m3" else 2)
        if case["op"] == "fork":   # table rows read and written, counts, and half a page copied for each copy
            n, held = case["rows"] * case["fan"], case["ctx"] // ps + 1
            return {"bytes": n * held * 4 * 3 + case["pages"] * 4 + n * page, "flops": n * held}
        held = min(case["pages"], -(-case["rows"] // case["fan"]) * (case["ctx"] // ps + 1))
        moved = held * (case["pages"] - held) // case["pages"]
        return {"bytes": moved * page * 2 + case["pages"] * 12 + case["rows"] * (case["ctx"] // ps + 1) * 8,
                "flops": case["pages"]}
    new, total = _lengths(case)
    wide = 2 if case["kv"] == "same" else 1
    if case["op"] == "append":
        n = sum(new) * Hkv * D * 2
        return {"bytes": n * (2 + wide), "flops": n}
    seen = [_seen(a, b, case["window"], case["sinks"]) for a, b in zip(new, total)]
    return {"bytes": sum(x[1] for x in seen) * Hkv * D * 2 * wide + sum(new) * case["Hq"] * (D * 4 + 4),
            "flops": sum(x[0] for x in seen) * case["Hq"] * D * 4}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, sequence by sequence; None for what is only moved."""
    if case["op"] in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    new, _ = _lengths(case)
    ps, Hkv, D = case["ps"], case["Hkv"], case["D"]
    f64 = torch.float64
    if case["op"] == "append":
        k, v = s["k"].to(f64), s["v"].to(f64)
        at = 0
        for b, n in enumerate(new):
            row = int(s["rows"][b])
            last = int(s["lens"][row])
            pos = torch.arange(last - n, last, device="cuda")
            page = s["table"][row].long()[pos // ps]
            for cache, x, sc in ((k, s["k_new"], s.get("k_scale")), (v, s["v_new"], s.get("v_scale"))):
                y = x[at:at + n].to(f64)
                if sc is not None:
                    y = (y / sc[0].to(f64)[:, None]).clamp(-448.0, 448.0)
                cache[0, page, :, pos % ps] = y
            at += n
        return k, v
    Hq = case["Hq"]
    G = Hq // Hkv
    q = s["q"].flatten(0, 1) if case["op"] == "decode" else s["q"]
    out = torch.zeros(q.shape, dtype=f64, device="cuda")
    lse = torch.full(q.shape[:2], NEG, dtype=f64, device="cuda")
    at = 0
    for b, n in enumerate(new):
        row = int(s["rows"][b])
        L = int(s["lens"][row])
        pages = s["table"][row, :-(-L // ps)].long()
        for g in range(Hkv):
            k = s["k"][0, pages, g].to(f64).reshape(-1, D)[:L]
            v = s["v"][0, pages, g].to(f64).reshape(-1, D)[:L]
            if s.get("k_scale") is not None:
                k, v = k * s["k_scale"][0, g].to(f64), v * s["v_scale"][0, g].to(f64)
            for h in range(g * G, (g + 1) * G):
                w = (q[at:at + n, h].to(f64) @ k.T) / D ** 0.5
                i = torch.arange(L - n, L, device="cuda")[:, None]
                j = torch.arange(L, device="cuda")[None]
                hidden = j > i
                if case["window"]:
                    hidden |= (j <= i - case["window"]) & (j >= case["sinks"])
                w = w.masked_fill(hidden, NEG)
                lse[at:at + n, h] = torch.logsumexp(w, 1)
                out[at:at + n, h] = torch.softmax(w, 1) @ v
        at += n
    shape = s["q"].shape
    return out.view(shape), lse.view(shape[:-1])
