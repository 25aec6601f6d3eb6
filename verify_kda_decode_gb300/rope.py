"""ctypes binding of libkda's rotary positions (include/kda.h): queries and keys turned by their positions, on their
own (``kda_rope``) or on their way into a paged cache (``kda_kv_append_rope``).

Argument checks and marshalling only, in the manner of ``paged.py``; the rules on streams and outputs there hold here.
A ``KdaRope`` holds the frequencies as fractions of a turn in 64-bit fixed point, made once on the host.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from fractions import Fraction
from typing import Optional, Sequence

import torch

from .kda import _call, _Copies, _lib, _need, _ptr, _stream
from .paged import _TYPES, KdaKvCache, _i32, _ints, _Layout, _plan, _rows, _tokens

_PI = Fraction(3141592653589793238462643383279502884197169399375106, 10 ** 51)


class _RopeDesc(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float)]


class _RopeLayout(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("src", _Layout), ("dst", _Layout)]


@dataclass
class KdaRope(_Copies):
    """How positions turn the pairs of a head (see kda_rope_desc in include/kda.h)."""
    turns: torch.Tensor        # int64 [rotary_dim / 2]: turns per position, in units of 2^-64 (modulo 2^64)
    interleaved: bool = False  # pairs (2 i, 2 i + 1) instead of (i, i + rotary_dim / 2)
    scale: float = 1.0         # what the turned elements are multiplied with

    @staticmethod
    def from_frequencies(frequencies: Sequence[float], interleaved: bool = False, scale: float = 1.0, device="cuda") -> "KdaRope":
        """Of `frequencies` in radians per position, one for each pair (floats, or a tensor that is read on the host)."""
        if isinstance(frequencies, torch.Tensor):
            frequencies = frequencies.double().cpu().tolist()
        turns = []
        for f in frequencies:
            if not math.isfinite(f):
                raise ValueError(f"frequency {f} is not finite")
            t = round(Fraction(f) / (2 * _PI) * (1 << 64)) % (1 << 64)
            turns.append(t - (1 << 64) if t >= 1 << 63 else t)
        return KdaRope(torch.tensor(turns, dtype=torch.int64, device=device), bool(interleaved), float(scale))

    @staticmethod
    def make(rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0, original_len: int = 4096,
             beta_fast: float = 32.0, beta_slow: float = 1.0, interleaved: bool = False, device="cuda") -> "KdaRope":
        """Frequencies base^(-2 i / rotary_dim), scaled for contexts `factor` times as long as trained:
        None; "linear" (positions divided by factor); "ntk" (a larger base, the slowest pair divided by factor); "yarn" (pairs
        that turn less than beta_slow times in original_len positions divided by factor, those above beta_fast kept, a ramp
        over the pairs between, and everything multiplied by 0.1 ln(factor) + 1; beta_slow is at most beta_fast)."""
        if rotary_dim < 2 or rotary_dim % 2:
            raise ValueError(f"rotary_dim={rotary_dim} must be even")
        if not (factor > 0 and math.isfinite(factor) and base > 1 and math.isfinite(base)):
            raise ValueError(f"factor={factor} must be positive and base={base} above 1")
        if scaling == "ntk":
            if rotary_dim < 4:
                raise ValueError('"ntk" needs rotary_dim >= 4')
            base *= factor ** (rotary_dim / (rotary_dim - 2))
        f = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
        scale = 1.0
        if scaling == "linear":
            f = [x / factor for x in f]
        elif scaling == "yarn":
            if not (0 < original_len < math.inf and 0 < beta_slow <= beta_fast < math.inf):
                raise ValueError(f"original_len={original_len}, beta_fast={beta_fast}, beta_slow={beta_slow}: each must be positive and finite, beta_slow at most beta_fast")

            def pair(turns):   # (fractional) pair that turns so many times
                return rotary_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))

            lo, hi = max(0, math.floor(pair(beta_fast))), min(rotary_dim - 1, math.ceil(pair(beta_slow)))
            keep = [1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rotary_dim // 2)]
            if pair(beta_slow) < 0:   # no pair turns so often: the ramp, which begins at pair 0 at the earliest, has no place
                keep = [0.0] * len(keep)
            f = [x * k + x / factor * (1.0 - k) for x, k in zip(f, keep)]
            scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        elif scaling not in (None, "ntk"):
            raise ValueError(f'scaling={scaling!r}: expected None, "linear", "ntk" or "yarn"')
        return KdaRope.from_frequencies(f, interleaved, scale, device)

    @property
    def device(self) -> torch.device:
        return self.turns.device

    @property
    def rotary_dim(self) -> int:
        return 2 * self.turns.shape[0]

    def __setattr__(self, name, value):
        # another value in a field: the struct that was built of it goes
        d = self.__dict__
        d[name] = value
        if not name.startswith("_"):
            d.pop("_c_struct", None)

    def c_struct(self) -> _RopeDesc:
        return self._struct()[0]

    def _struct(self):
        """(struct, reference to it), checked and built once while the same storage is attached."""
        d = self.__dict__
        cached = d.get("_c_struct")
        if cached is not None and cached[2] == self.turns.data_ptr():
            return cached
        if not isinstance(self.turns, torch.Tensor) or self.turns.dim() != 1:
            raise ValueError("turns must be an int64 tensor [rotary_dim / 2]")
        _need(self.turns, "turns", torch.int64, self.turns.shape, self.turns.device)
        st = _RopeDesc(_ptr(self.turns), _i32(self.rotary_dim, "rotary_dim"), int(bool(self.interleaved)), float(self.scale))
        d["_c_struct"] = cached = (st, ctypes.byref(st), self.turns.data_ptr())
        return cached


def _same_device(rope: KdaRope, dev) -> None:
    if rope.turns.device != dev:
        raise ValueError(f"rope: on {rope.turns.device}, expected {dev}")


def _heads(t: torch.Tensor, name: str, D: int, dev) -> _Layout:
    """Layout of [B, T, heads, D] or [N, heads, D] of this head dim: any strides, the last dimension contiguous."""
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name}: dtype {t.dtype}, expected bfloat16 or float16")
    n = t.shape
    if len(n) not in (3, 4) or n[-1] != D:
        raise ValueError(f"{name}: shape {tuple(n)}, expected [B, T, heads, {D}] or [N, heads, {D}]")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, expected {dev}")
    _i32(max(n), f"{name}: size")
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"{name}: its last dimension must be contiguous")
    # a dimension of one element has no stride to speak of
    return _Layout(_TYPES[t.dtype], 0 if len(n) == 3 or n[0] == 1 else st[0], 0 if n[-3] == 1 else st[-3], 0 if n[-2] == 1 else st[-2])


def _form(out, name: str):
    """What the plan of a call into the caller's tensor goes by."""
    if not isinstance(out, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return out.dtype, out.device, out.shape, out.stride()


def _turned(t, out, name: str, D: int, dev) -> _RopeLayout:
    """Layouts of t and of its turned copy; out None: a contiguous tensor that the call makes."""
    src = _heads(t, name, D, dev)
    if out is None:
        H, T = t.shape[-2], t.shape[-3]
        dst = _Layout(src.dtype, 0 if t.dim() == 3 or t.shape[0] == 1 else T * H * D, 0 if T == 1 else H * D, 0 if H == 1 else D)
    elif out.shape != t.shape or out.dtype != t.dtype:
        raise ValueError(f"{name}_out: {out.dtype} {tuple(out.shape)}, expected {t.dtype} {tuple(t.shape)}")
    else:
        dst = _heads(out, name + "_out", D, dev)
    return _RopeLayout(t.shape[-2], src, dst)


def kda_rope(rope: KdaRope, positions, q, k=None, q_out=None, k_out=None, stream=None):
    """Turns q [B, T, Hq, D] (or [N, Hq, D]), and k [B, T, Hk, D] (or [N, Hk, D]) with it, by positions int32 [B, T] (or [N]);
    negative ones turn back.  q and k may have any strides in multiples of 8 elements, their last dimension contiguous; q_out
    and k_out too, and may be q and k themselves.  Returns the turned q, or (q, k) where k is given."""
    if not isinstance(q, torch.Tensor) or (k is not None and not isinstance(k, torch.Tensor)):
        raise TypeError("q and k must be torch.Tensors")
    dev = q.device
    _same_device(rope, dev)
    ref = rope._struct()[1]
    key = ("rope", dev, q.dtype, q.shape, q.stride())
    if q_out is not None:
        key += ("q",) + _form(q_out, "q_out")
    if k is not None:
        key += (k.dtype, k.device, k.shape, k.stride())
        if k_out is not None:
            key += ("k",) + _form(k_out, "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")

    def make():
        D = q.shape[-1] if q.dim() else 0
        ql = _turned(q, q_out, "q", D, dev)
        kl = None if k is None else _turned(k, k_out, "k", D, dev)
        if k is not None and (k.shape[:-2] != q.shape[:-2] or k.dtype != q.dtype):
            raise ValueError(f"q and k: {q.dtype} {tuple(q.shape)} and {k.dtype} {tuple(k.shape)} are not of the same tokens and type")
        B, T = (1, q.shape[0]) if q.dim() == 3 else q.shape[:2]
        return q.shape[:-2], D, B, T, ctypes.byref(ql), None if kl is None else ctypes.byref(kl)

    tokens, D, B, T, ql, kl = _plan(rope, key, make)
    _need(positions, "positions", torch.int32, tokens, dev)
    # outputs last: an allocation right behind the last call's launch waits for it (a call of one token 16.3 us, like this 13.8)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if k is not None and k_out is None:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
    _call(dev, _lib.kda_rope, ref, D, positions.data_ptr(), B, T, ql, q.data_ptr(), q_out.data_ptr(), kl,
          None if k is None else k.data_ptr(), None if k is None else k_out.data_ptr(), _stream(stream, dev))
    return q_out if k is None else (q_out, k_out)


def kda_kv_append_rope(cache: KdaKvCache, layer: int, rows, rope: KdaRope, q, k, v, cu_seqlens=None, n_tokens=None, q_out=None,
                       stream=None):
    """kda_kv_append of keys that are turned by their positions in the row on the way, with the new tokens' queries: q
    [B, T, Hq, D], or [N, Hq, D] packed as k and v are, in their type; None: keys alone.  q_out: as in kda_rope.  Returns the
    turned q (None without q); tokens that the append leaves out leave theirs as it was in q_out."""
    _, st, _, dev = cache._struct()
    _same_device(rope, dev)
    ref = rope._struct()[1]
    pr, B = _rows(rows, dev)
    for name, t in (("k", k), ("v", v)) + ((("q", q),) if q is not None else ()):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    key = ("append_rope", B, cu_seqlens is None, k.dtype, v.dtype, k.device, v.device, k.shape, v.shape, k.stride(), v.stride())
    if q is not None:
        key += (q.dtype, q.device, q.shape, q.stride())
        if q_out is not None:
            key += _form(q_out, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")

    def make():
        packed = k.dim() == 3
        kl, vl = _tokens(k, "k", packed, cache.Hkv, cache), _tokens(v, "v", packed, cache.Hkv, cache)
        ql = None
        if k.shape != v.shape:
            raise ValueError(f"k and v have shapes {tuple(k.shape)} and {tuple(v.shape)}")
        if q is not None:
            if q.shape[:-2] != k.shape[:-2] or q.dtype != k.dtype:
                raise ValueError(f"q and k: {q.dtype} {tuple(q.shape)} and {k.dtype} {tuple(k.shape)} are not of the same tokens and type")
            ql = _turned(q, q_out, "q", cache.head_dim, dev)
        if cu_seqlens is not None:
            if not packed:
                raise ValueError("cu_seqlens goes with packed q, k and v [N, heads, D]")
            T = k.shape[0]
        elif packed:
            if B and k.shape[0] % B:
                raise ValueError(f"{k.shape[0]} packed tokens are no multiple of {B} rows: pass cu_seqlens")
            T = k.shape[0] // B if B else 0
            for x in (kl, vl) + (() if ql is None else (ql.src, ql.dst)):
                x.seq_stride = T * x.token_stride
        else:
            if k.shape[0] != B:
                raise ValueError(f"k: {k.shape[0]} sequences, rows has {B}")
            T = k.shape[1]
        return T, None if ql is None else ctypes.byref(ql), ctypes.byref(kl), ctypes.byref(vl)

    T, ql, kl, vl = _plan(cache, key, make)
    pc = None if cu_seqlens is None else _ints(cu_seqlens, "cu_seqlens", B + 1, dev)
    pn = None if n_tokens is None else _ints(n_tokens, "n_tokens", B, dev)
    if q is not None and q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    _call(dev, _lib.kda_kv_append_rope, st, _i32(layer, "layer"), ref, pr, B, T, pn, pc, ql, None if q is None else q.data_ptr(),
          None if q is None else q_out.data_ptr(), k.data_ptr(), kl, v.data_ptr(), vl, _stream(stream, dev))
    return q_out
