"""Plain references of 4-bit caches (E2M1 codes, an E4M3 scale for each 16 elements) and of rotary positions, on the CPU."""
from __future__ import annotations

import torch

F64 = torch.float64
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=F64)


def nearest_code(q):
    """E2M1 codes of q: the nearest, of two the even one, 6 at most; the sign in the fourth bit."""
    a = q.abs().to(F64)
    code = torch.zeros(q.shape, dtype=torch.int64)
    for i, t in enumerate(((GRID[1:] + GRID[:-1]) / 2).tolist()):   # the border between codes i and i + 1
        code += (a >= t) if i % 2 else (a > t)
    return code + 8 * torch.signbit(q).long()


def quantize(x, scale):
    """x [..., D] in 32 bits, divided by `scale`, -> (codes [..., D], block scales [..., D / 16] as E4M3), each step an IEEE operation
    in 32 bits rounded as the format says."""
    assert x.dtype == torch.float32
    y = (x / scale).unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1) / 6.0).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    return nearest_code(y / s.float()[..., None]).flatten(-2), s


def values(codes, s, scale):
    """What codes and block scales stand for, in 64 bits."""
    v = GRID[codes & 7] * (1 - 2 * (codes >> 3)).to(F64)
    return v * s.to(F64).repeat_interleave(16, -1) * scale


def packed(codes, s):
    """codes [..., tokens, D], s [..., tokens, D / 16] of whole pages -> bytes [..., tokens, D / 2 + D / 16] as a page's head holds them."""
    b = (codes[..., 0::2] | codes[..., 1::2] << 4).to(torch.uint8).flatten(-2)
    raw = torch.cat([b, s.view(torch.uint8).flatten(-2)], -1)
    ps = codes.shape[-2]
    return raw.unflatten(-1, (ps, -1))


def unpacked(raw, D):
    """Bytes [..., page size, D / 2 + D / 16] -> (codes [..., page size, D], block scales [..., page size, D / 16])."""
    ps = raw.shape[-2]
    flat = raw.flatten(-2)
    b = flat[..., :ps * D // 2].unflatten(-1, (ps, D // 2)).long()
    s = flat[..., ps * D // 2:].contiguous().view(torch.float8_e4m3fn).unflatten(-1, (ps, D // 16))
    return torch.stack([b & 15, b >> 4], -1).flatten(-2), s


def make_cache4(K, lens, Hkv, D, ps, seed=0, layers=1, layer=0, extra_pages=3, extra_rows=2, spread=1.0):
    """make_cache of paged_ref.py with 4 bits: rows of `lens` tokens in randomly placed pages of `layer`; whatever no row holds
    has NaN for its block scales."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // ps) for n in lens]
    pages, rows, width = sum(counts) + extra_pages, len(lens) + extra_rows, max(counts + [1]) + 1
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((rows, width), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    codes = [torch.randint(0, 16, (layers, pages, Hkv, ps, D), generator=g) for _ in range(2)]
    scales = [torch.full((layers, pages, Hkv, ps, D // 16), float("nan")).to(torch.float8_e4m3fn) for _ in range(2)]
    ls = [0.3 + 0.4 * torch.rand(layers, Hkv, generator=g) for _ in range(2)]
    dense, at = [], 0
    for r, n in enumerate(lens):
        both = []
        for c, s, l in zip(codes, scales, ls):
            x = torch.randn(n, Hkv, D, generator=g) * torch.exp(spread * torch.randn(n, Hkv, 1, generator=g))
            qc, qs = quantize(x, l[layer][:, None])
            both.append((qc, qs))
            for j in range(counts[r]):
                page, part = order[at + j], slice(j * ps, min(n, (j + 1) * ps))
                m = part.stop - part.start
                c[layer, page, :, :m] = qc[part].transpose(0, 1)
                s[layer, page, :, :m] = qs[part].transpose(0, 1)
        for j in range(counts[r]):
            table[r, j] = order[at + j]
            refs[order[at + j]] += 1
        at += counts[r]
        dense.append(tuple(values(c, s, l[layer].to(F64)[:, None]) for (c, s), l in zip(both, ls)))
    seq = torch.zeros(rows, dtype=torch.int32)
    seq[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
    cache = K.KdaKvCache(k=packed(codes[0], scales[0]).cuda(), v=packed(codes[1], scales[1]).cuda(), page_table=table.cuda(),
                         seq_lens=seq.cuda(), page_refs=refs.cuda(), k_scale=ls[0].cuda(), v_scale=ls[1].cuda())
    return cache, dense


def token_codes(cache, layer, row, pos):
    """(codes [2, Hkv, D], block scales [2, Hkv, D / 16]) of a row's token, keys then values, on the CPU."""
    ps = cache.k.shape[3]
    page = int(cache.page_table[row, pos // ps])
    got = [unpacked(x[layer, page].cpu(), cache.head_dim) for x in (cache.k, cache.v)]
    return torch.stack([c[:, pos % ps] for c, _ in got]), torch.stack([s[:, pos % ps].float() for _, s in got])


def turned(x, pos, freqs, interleaved=False, scale=1.0):
    """x [N, H, D] turned by pos [N] times freqs (radians per position, as floats), by complex numbers in 64 bits."""
    rot = 2 * len(freqs)
    angle = pos.to(F64)[:, None] * torch.tensor(freqs, dtype=F64)
    unit = torch.polar(torch.full_like(angle, scale), angle)[:, None]
    head = x.to(F64)[..., :rot]
    if interleaved:
        head = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * unit).flatten(-2)
    else:
        z = torch.complex(*(t.contiguous() for t in head.chunk(2, -1))) * unit
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, x.to(F64)[..., rot:]], -1)


def turn_error(x, rot, interleaved=False, scale=1.0):
    """How far FP32 may be off before the output's own rounding, per element of x [N, H, D]: the angle's 32 bits (2^-26 of a turn
    by the conversion to FP32, 2^-33 by the cut: under 2^-23 of cosine and sine), one unit in the last place of sincospif
    (2^-24 at most) and the roundings of the products with the scale, of one product and of the sum (2^-24 each of their
    size): 2^-22 of |a| + |b| in all."""
    mag = x.to(F64).abs()
    head = mag[..., :rot]
    both = head[..., 0::2] + head[..., 1::2] if interleaved else head[..., :rot // 2] + head[..., rot // 2:]
    both = both.repeat_interleave(2, -1) if interleaved else torch.cat([both, both], -1)
    return torch.cat([both * 2.0 ** -22 * abs(scale), torch.zeros_like(mag[..., rot:])], -1)
