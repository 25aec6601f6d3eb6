"""A small hybrid model served end to end: KDA mixer layers with softmax-attention layers between them.

Random weights; the point is how the calls go together.  The attention layers may rotate queries and keys by their
positions (on the keys' way into the cache), and the cache may hold 16, 8 or 4 bits.  Two prompts are prefilled in one packed call,
each is forked into two samples, the samples decode token by token, then verify drafts of which some
are accepted, and finish: their pages are given back and the cache is closed up.  At the end every
sample's tokens are run again as one prompt, and the two ways have to agree.

    python examples/hybrid_decode.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import verify_kda_decode_gb300 as K  # noqa: E402

BF = torch.bfloat16


class Hybrid:
    """`kinds`: "kda" for a KDA mixer layer, a window (0 = none) for a softmax-attention layer; `rotary_dim`: elements of a head
    that the attention layers rotate (0: none)."""

    def __init__(self, kinds=("kda", 0, "kda", 64), width=256, H=2, Hq=4, Hkv=2, D=64, seed=0, rows=16, pages=64, ps=16, cache_dtype=BF,
                 rotary_dim=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s, std=None: (torch.randn(*s, device="cuda", generator=g) * (std or s[0] ** -0.5)).to(BF)
        self.kinds, self.width, self.H, self.Hq, self.Hkv, self.D = kinds, width, H, Hq, Hkv, D
        self.parts = [128 * H, 128 * H, 128 * H, 128, H, 128 * H]   # q, k, v, f_a, beta, gate
        self.layers, self.pools = [], []
        for kind in kinds:
            if kind == "kda":
                mixer = K.KdaLayer(W_fb=w(H * 128, 128, std=0.02), A_log=torch.zeros(H, device="cuda"), dt_bias=torch.zeros(H * 128, device="cuda"),
                                   conv_w=w(3, H * 128, 4, std=0.3), norm_w=torch.ones(128, device="cuda"))
                self.layers.append((w(width, sum(self.parts)), mixer, w(H * 128, width)))
                self.pools.append(K.KdaPool.zeros(rows, H))
            else:
                self.layers.append((w(width, (Hq + 2 * Hkv) * D), kind, w(Hq * D, width)))
                self.pools.append(None)
        self.cache = K.KdaKvCache.zeros(sum(k != "kda" for k in kinds), pages, Hkv, rows, 12, ps, D, dtype=cache_dtype)
        if cache_dtype == torch.float8_e4m3fn:
            self.cache.k_scale.fill_(0.02)
            self.cache.v_scale.fill_(0.02)
        self.rope = K.KdaRope.make(rotary_dim, scaling="yarn", factor=4.0, original_len=64) if rotary_dim else None

    def _norm(self, x):
        return torch.nn.functional.rms_norm(x.float(), (self.width,)).to(BF)

    def _run(self, x, rows, mixer_call, attn_call, records=None):
        at = 0
        for kind, (w_in, layer, w_out), pool in zip(self.kinds, self.layers, self.pools):
            y = self._norm(x) @ w_in
            if kind == "kda":
                ins = [t.contiguous() for t in y.split(self.parts, -1)]
                o = mixer_call(layer, pool, rows, *ins)
                if records is not None:
                    records.append((pool, o[1], o[2]))
                    o = o[0]
            else:
                q, k, v = (t.unflatten(-1, (-1, self.D)) for t in y.split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], -1))
                o = attn_call(at, q, k, v, kind).flatten(-2)
                at += 1
            x = x + o @ w_out
        return x

    def _append(self, layer, rows, q, k, v, cu=None):
        """New keys and values into the cache; returns the queries that attend."""
        if self.rope is None:
            K.kda_kv_append(self.cache, layer, rows, k, v, cu_seqlens=cu)
            return q
        return K.kda_kv_append_rope(self.cache, layer, rows, self.rope, q, k, v, cu_seqlens=cu)

    def prefill(self, x, rows, cu, lens):
        """Packed prompts x [tokens, width], sequence b in row rows[b]."""
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        K.kda_kv_extend(self.cache, rows, n)

        def attn(layer, q, k, v, window):
            q = self._append(layer, rows, q, k, v, cu)
            return K.kda_attn_prefill(self.cache, layer, rows, cu, max(lens), q, window=window, sinks=4)

        return self._run(x, rows, lambda la, p, r, *i: K.kda_prefill_varlen(la, p, r, cu, max(lens), *i), attn)

    def _attn_step(self, rows):
        def attn(layer, q, k, v, window):
            q, k, v = (t if t.dim() == 4 else t[:, None] for t in (q, k, v))
            q = self._append(layer, rows, q, k, v)
            return K.kda_attn_decode(self.cache, layer, rows, q, window=window, sinks=4)

        return attn

    def decode(self, x, rows):
        """One token of each row, x [B, width]."""
        K.kda_kv_extend(self.cache, rows, 1)
        attn = self._attn_step(rows)
        return self._run(x, rows, K.kda_decode, lambda *a: attn(*a)[:, 0])

    def verify(self, x, rows, accepted):
        """T drafts of each row, x [B, T, width], of which accepted[b] stay."""
        B, T = x.shape[:2]
        K.kda_kv_extend(self.cache, rows, T)
        records = []
        out = self._run(x, rows, K.kda_verify, self._attn_step(rows), records)
        for pool, state, conv in records:
            K.kda_commit(pool, rows, accepted, state, conv)
        K.kda_kv_truncate(self.cache, rows, self.cache.seq_lens[rows.long()] - T + accepted)
        return out

    def fork(self, src, dst):
        K.kda_kv_fork(self.cache, src, dst)
        for pool in self.pools:
            if pool is not None:
                pool.state[dst.long()] = pool.state[src.long()]
                pool.conv_state[dst.long()] = pool.conv_state[src.long()]

    def free(self, rows):
        K.kda_kv_truncate(self.cache, rows, torch.zeros_like(rows))
        for pool in self.pools:
            if pool is not None:
                pool.state[rows.long()] = 0
                pool.conv_state[rows.long()] = 0

    def errors(self):
        return [K.kda_kv_get_error(self.cache)] + [K.kda_get_error(p) for p in self.pools if p is not None]


def serve(model, seed=1, lens=(37, 70), steps=5, T=4):
    """Runs the scenario of this file; returns the largest difference between a sample's step outputs and the
    same tokens run as one prompt, relative to the largest output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = lambda *s: torch.randn(*s, model.width, device="cuda", generator=g).to(BF)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    prompts = [x(n) for n in lens]
    cu = i32([0] + [sum(lens[:i + 1]) for i in range(len(lens))])
    model.prefill(torch.cat(prompts), i32([0, 1]), cu, list(lens))
    model.fork(i32([0, 1]), i32([2, 3]))           # two samples of each prompt
    rows = i32([0, 1, 2, 3])
    fed = [[prompts[r % 2]] for r in range(4)]
    got = [[] for _ in range(4)]
    for _ in range(steps):
        tok = x(4)
        out = model.decode(tok, rows)
        for r in range(4):
            fed[r].append(tok[r:r + 1])
            got[r].append(out[r:r + 1])
    drafts, accepted = x(4, T), [0, 1, T, 2]
    out = model.verify(drafts, rows, i32(accepted))
    for r, n in enumerate(accepted):
        fed[r].append(drafts[r, :n])
        got[r].append(out[r, :n])
    tok = x(4)                                     # and on from what was accepted
    out = model.decode(tok, rows)
    for r in range(4):
        fed[r].append(tok[r:r + 1])
        got[r].append(out[r:r + 1])
    model.free(i32([0, 1]))
    K.kda_kv_compact(model.cache)                  # the other two move down
    tok = x(2)
    out = model.decode(tok, i32([2, 3]))
    for i, r in enumerate((2, 3)):
        fed[r].append(tok[i:i + 1])
        got[r].append(out[i:i + 1])
    model.free(i32([2, 3]))
    assert int(model.cache.page_refs.sum()) == 0 and not any(model.errors()), model.errors()
    # every sample again, as one prompt
    seqs = [torch.cat(f) for f in fed]
    n = [s.shape[0] for s in seqs]
    cu = i32([0] + [sum(n[:i + 1]) for i in range(4)])
    whole = model.prefill(torch.cat(seqs), i32([4, 5, 6, 7]), cu, n)
    assert not any(model.errors()), model.errors()
    worst = 0.0
    for r in range(4):
        a = torch.cat(got[r]).float()
        b = whole[int(cu[r + 1]) - a.shape[0]:int(cu[r + 1])].float()
        worst = max(worst, float((a - b).abs().max() / b.abs().max()))
    return worst


if __name__ == "__main__":
    for name, kw in (("bfloat16", dict()), ("E4M3", dict(cache_dtype=torch.float8_e4m3fn)), ("bfloat16, rotated", dict(rotary_dim=32)),
                     ("4-bit, rotated", dict(cache_dtype=torch.uint8, rotary_dim=64))):
        print("%s cache: step by step against one prompt, largest difference %.2g of the largest output" % (name, serve(Hybrid(**kw))))
