"""Plain 64-bit references of the paged cache's operators, on the CPU, and the tolerances that go with them."""
from __future__ import annotations

import math
import random

import torch

F64 = torch.float64
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative


def make_cache(K, lens, Hkv, D, ps, dtype, seed=0, layers=1, layer=0, extra_pages=3, extra_rows=2, garbage=float("nan")):
    """A cache whose rows hold `lens` tokens in randomly placed pages of `layer`; whatever no row holds is
    `garbage`.  Returns it with the dense values [rows][len, Hkv, D] in 64 bits (scales applied)."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // ps) for n in lens]
    pages, rows, width = sum(counts) + extra_pages, len(lens) + extra_rows, max(counts + [1]) + 1
    fp8 = dtype == torch.float8_e4m3fn
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((rows, width), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    k = torch.full((layers, pages, Hkv, ps, D), garbage)
    v = k.clone()
    ks = 0.01 + 0.02 * torch.rand(layers, Hkv, generator=g) if fp8 else None
    vs = 0.01 + 0.02 * torch.rand(layers, Hkv, generator=g) if fp8 else None
    dense = []
    at = 0
    for r, n in enumerate(lens):
        kk, vv = (torch.randn(n, Hkv, D, generator=g) * (60 if fp8 else 1) for _ in range(2))
        if fp8:
            kk, vv = kk.clamp(-448, 448), vv.clamp(-448, 448)
        kk, vv = kk.to(dtype).float(), vv.to(dtype).float()
        for j in range(counts[r]):
            page = order[at]
            at += 1
            table[r, j] = page
            refs[page] += 1
            part = slice(j * ps, min(n, (j + 1) * ps))
            m = part.stop - part.start
            k[layer, page, :, :m] = kk[part].transpose(0, 1)
            v[layer, page, :, :m] = vv[part].transpose(0, 1)
        if fp8:
            dense.append((kk.to(F64) * ks[layer].to(F64)[:, None], vv.to(F64) * vs[layer].to(F64)[:, None]))
        else:
            dense.append((kk.to(F64), vv.to(F64)))
    seq = torch.zeros(rows, dtype=torch.int32)
    seq[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
    dev = lambda t: None if t is None else t.cuda()
    cache = K.KdaKvCache(k=k.to(dtype).cuda(), v=v.to(dtype).cuda(), page_table=table.cuda(), seq_lens=seq.cuda(),
                         page_refs=refs.cuda(), k_scale=dev(ks), v_scale=dev(vs))
    return cache, dense


def attention(q, k, v, length, scale, window, sinks):
    """q [n, Hq, D] at positions length - n .. length - 1 over k, v [length, Hkv, D], all in 64 bits.
    Returns out, lse, the attention-weighted |v| and the largest sum |q k| scale of a row."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1] if k.shape[0] else 1
    out, lse = torch.zeros(n, Hq, D, dtype=F64), torch.full((n, Hq), -math.inf, dtype=F64)
    mag, size = torch.zeros(n, Hq, D, dtype=F64), torch.zeros(n, Hq, dtype=F64)
    j = torch.arange(length)
    for t in range(n):
        p = length - n + t
        see = j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
        if p < 0 or not see.any():
            continue
        kk = k[see].repeat_interleave(G, 1)          # [keys, Hq, D]
        vv = v[see].repeat_interleave(G, 1)
        s = torch.einsum("hd,jhd->hj", q[t], kk) * scale
        lse[t] = torch.logsumexp(s, 1)
        w = torch.softmax(s, 1)
        out[t] = torch.einsum("hj,jhd->hd", w, vv)
        mag[t] = torch.einsum("hj,jhd->hd", w, vv.abs())
        size[t] = (torch.einsum("hd,jhd->hj", q[t].abs(), kk.abs()) * scale).amax(1)
    return out, lse, mag, size


def check_attention(got, got_lse, ref, dtype, keys):
    """The tolerance counts roundings: the output's own and that of each P to 16 bits (half a step each, the
    latter weighted by |v|), and FP32 arithmetic: D sums of the scores' products (truncated to 2^-23 of the
    sum of their magnitudes), exponentials and sums to 2^-22 and 2^-24 a term."""
    out, lse, mag, size = ref
    D = out.shape[-1]
    s_err = D * 2.0 ** -23 * size + 2.0 ** -20          # absolute error of a score, and of the exponential
    l_err = keys * 2.0 ** -24 + 2.0 ** -20
    tol = 1.01 * (EPS[dtype] * (out.abs() + mag) + (2 * s_err + 2 * l_err)[..., None] * mag) + 2.0 ** -24
    err = (got.to(F64).cpu() - out).abs()
    assert not torch.isnan(got).any()
    assert (err <= tol).all(), "off by up to %.3g of the tolerance" % (err / tol).max()
    if got_lse is not None:
        g = got_lse.to(F64).cpu()
        none = torch.isinf(lse)
        assert torch.equal(none, torch.isinf(g) & (g < 0))
        bad = (g - lse).abs()[~none]
        lim = (s_err + l_err + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0))[~none]
        assert (bad <= lim).all(), "lse off by up to %.3g of the tolerance" % (bad / lim).max()


class PageModel:
    """The page calls in plain Python: what tables, lengths, counts and contents have to be."""

    def __init__(self, rows, width, pages, ps, layers=1):
        self.ps, self.width, self.pages, self.layers = ps, width, pages, layers
        self.table = [[] for _ in range(rows)]
        self.lens = [0] * rows
        self.refs = [0] * pages
        self.data = [[[None] * ps for _ in range(pages)] for _ in range(layers)]
        self.err = 0

    def need(self, n):
        return -(-n // self.ps)

    def _distinct(self, rows):
        return [0 <= r < len(self.lens) and rows.count(r) == 1 for r in rows]

    def extend(self, rows, n):
        ok, want = self._distinct(rows), []
        for r, m, good in zip(rows, n, ok):
            if not good:
                self.err |= 0x1
                want.append(None)
            elif m < 0:
                self.err |= 0x10
                want.append(None)
            elif self.lens[r] + m > self.width * self.ps:
                self.err |= 0x80
                want.append(None)
            else:
                copy = m > 0 and self.lens[r] % self.ps != 0 and self.refs[self.table[r][-1]] > 1
                want.append((copy, self.need(self.lens[r] + m) - self.need(self.lens[r]) + copy))
        free = [p for p in range(self.pages) if self.refs[p] == 0]
        off, moves = 0, []
        for r, m, w in zip(rows, n, want):
            if w is None:
                continue
            copy, count = w
            if count and off + count > len(free):
                self.err |= 0x80
            else:
                ids = free[off:off + count]
                if copy:
                    old, new = self.table[r][-1], ids.pop(0)
                    moves.append((old, new, self.lens[r] % self.ps))
                    self.refs[old] -= 1
                    self.refs[new] = 1
                    self.table[r][-1] = new
                for p in ids:
                    self.refs[p] = 1
                self.table[r] += ids
                self.lens[r] += m
            off += count
        for old, new, m in moves:
            for d in self.data:
                d[new][:m] = d[old][:m]

    def truncate(self, rows, lens):
        for r, m, good in zip(rows, lens, self._distinct(rows)):
            if not good:
                self.err |= 0x1
            elif m < 0 or m > self.lens[r]:
                self.err |= 0x20
            else:
                for p in self.table[r][self.need(m):]:
                    self.refs[p] -= 1
                self.table[r] = self.table[r][:self.need(m)]
                self.lens[r] = m

    def fork(self, src, dst):
        ok = self._distinct(dst)
        for s, d, good in zip(src, dst, ok):
            if not good or not 0 <= s < len(self.lens) or d in src:
                self.err |= 0x1
                continue
            for p in self.table[d]:
                self.refs[p] -= 1
            self.table[d] = list(self.table[s])
            for p in self.table[d]:
                self.refs[p] += 1
            self.lens[d] = self.lens[s]

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        high = [p for p in range(n, self.pages) if self.refs[p]]
        low = [p for p in range(n) if not self.refs[p]]
        remap = [p if self.refs[p] else -1 for p in range(self.pages)]
        for a, b in zip(high, low):
            remap[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
            for d in self.data:
                d[b] = list(d[a])
        self.table = [[remap[p] for p in t] for t in self.table]
        return remap

    def write(self, layer, row, pos, value):
        self.data[layer][self.table[row][pos // self.ps]][pos % self.ps] = value


def spread(n, most, seed):
    r = random.Random(seed)
    return [r.choice([1, 15, 16, 17, 63, 64, 65, r.randint(1, most), most]) for _ in range(n)]
