"""ctypes binding of libkda's paged key-value cache and the attention that reads it (include/kda.h).

Argument checks and marshalling only, in the manner of ``kda.py``: tensors are torch CUDA tensors,
calls run on the current stream of the cache's device with that device current.  A cache's own
workspaces are made and cleared with it, before its constructor returns: its calls may run on any
stream and be captured from the first one on.  Calls on one cache that may overlap on the GPU (two
streams without an order between them) have to pass workspaces of their own.  Outputs that a call
makes itself belong to the current stream: where ``stream`` names another one, order it after the
current one first, or pass ``out`` (``lse``, ``remap``).
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Tuple, Union

import torch

from .kda import (KDA_DEVERR_TIMEOUT, KDA_ERR_DEVICE, KDA_OK, KDA_T_BF16, KDA_T_E2M1, KDA_T_E4M3, KDA_T_F16, _call, _Copies, _lib, _need, _ptr, _raise,
                  _stream)

# of a cache; uint8 is the storage of a 4-bit one
_TYPES = {torch.bfloat16: KDA_T_BF16, torch.float16: KDA_T_F16, torch.float8_e4m3fn: KDA_T_E4M3, torch.uint8: KDA_T_E2M1}
_CODES = (torch.float8_e4m3fn, torch.uint8)


class _Cache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("kv_dtype", ctypes.c_int32),
        ("num_layers", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("rows", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("page_refs", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("err_word", ctypes.c_void_p),
    ]


class _Layout(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("seq_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _Desc(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("scale", ctypes.c_float), ("window", ctypes.c_int32),
                ("sinks", ctypes.c_int32), ("q", _Layout)]


@dataclass
class KdaKvCache(_Copies):
    """Caller-owned paged cache (see kda_kv_cache in include/kda.h).

    A 4-bit cache (E2M1 codes with an E4M3 scale for each 16 elements) is held as uint8 [layers, pages, Hkv, page size,
    D / 2 + D / 16]: the bytes of a page's head are those of all its codes and then those of all its block scales."""
    k: torch.Tensor            # bf16, f16 or float8_e4m3fn [layers, pages, Hkv, page size, D], or uint8 as above
    v: torch.Tensor            # like k
    page_table: torch.Tensor   # int32 [rows, max_pages], -1 where there is no page
    seq_lens: torch.Tensor     # int32 [rows]
    page_refs: torch.Tensor    # int32 [pages]: table entries that name each page
    k_scale: Optional[torch.Tensor] = None   # f32 [layers, Hkv] with float8_e4m3fn and uint8
    v_scale: Optional[torch.Tensor] = None
    err_word: Optional[torch.Tensor] = None  # int32 [1], zeroed; made here if not given

    def __post_init__(self):
        if self.err_word is None:
            self.err_word = torch.zeros(1, dtype=torch.int32, device=self.k.device)
        self._make_workspaces()

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._make_workspaces()   # a copy's own, as a new cache's

    @staticmethod
    def zeros(layers: int, num_pages: int, Hkv: int, rows: int, max_pages: int, page_size: int = 64,
              head_dim: int = 128, dtype=torch.bfloat16, device="cuda", k_scale=None, v_scale=None) -> "KdaKvCache":
        """An empty cache; with float8_e4m3fn and uint8 (4 bits) the scales are ones unless given."""
        shape = (layers, num_pages, Hkv, page_size, head_dim // 2 + head_dim // 16 if dtype == torch.uint8 else head_dim)
        if dtype in _CODES:
            k_scale = torch.ones(layers, Hkv, device=device) if k_scale is None else k_scale
            v_scale = torch.ones(layers, Hkv, device=device) if v_scale is None else v_scale
        raw = torch.uint8 if dtype == torch.float8_e4m3fn else dtype
        return KdaKvCache(
            k=torch.zeros(shape, dtype=raw, device=device).view(dtype), v=torch.zeros(shape, dtype=raw, device=device).view(dtype),
            page_table=torch.full((rows, max_pages), -1, dtype=torch.int32, device=device),
            seq_lens=torch.zeros(rows, dtype=torch.int32, device=device),
            page_refs=torch.zeros(num_pages, dtype=torch.int32, device=device), k_scale=k_scale, v_scale=v_scale)

    @property
    def device(self) -> torch.device:
        return self.k.device

    @property
    def Hkv(self) -> int:
        return self.k.shape[2]

    @property
    def head_dim(self) -> int:
        return self.k.shape[4] * 16 // 9 if self.k.dtype == torch.uint8 else self.k.shape[4]

    @property
    def num_pages(self) -> int:
        return self.k.shape[1]

    def __setattr__(self, name, value):
        # another tensor in a field: the struct and what was checked against it go
        d = self.__dict__
        d[name] = value
        if not name.startswith("_"):
            for k in ("_c_struct", "_plans"):
                d.pop(k, None)

    def c_struct(self) -> _Cache:
        return self._struct()[0]

    def _struct(self):
        """(struct, reference to it), checked and built once while the same storages are attached."""
        d = self.__dict__
        ptrs = (self.k.data_ptr(), self.v.data_ptr(), self.page_table.data_ptr(), self.seq_lens.data_ptr(),
                self.page_refs.data_ptr(), self.err_word.data_ptr(),
                self.k_scale.data_ptr() if self.k_scale is not None else 0, self.v_scale.data_ptr() if self.v_scale is not None else 0)
        cached = d.get("_c_struct")
        if cached is not None and cached[2] == ptrs:
            return cached
        if self.k.dtype not in _TYPES:
            raise TypeError(f"k: dtype {self.k.dtype}, expected bfloat16, float16, float8_e4m3fn or uint8 (4 bits)")
        if self.k.dim() != 5:
            raise ValueError(f"k: shape {tuple(self.k.shape)}, expected [layers, pages, Hkv, page size, D]")
        dev = self.k.device
        layers, pages, Hkv, ps, D = self.k.shape
        if self.k.dtype == torch.uint8:
            if D % 9:
                raise ValueError(f"k: shape {tuple(self.k.shape)}, a 4-bit cache has D / 2 + D / 16 bytes for each token")
            D = self.head_dim
        _need(self.k, "k", self.k.dtype, self.k.shape, dev)
        _need(self.v, "v", self.k.dtype, self.k.shape, dev)
        if self.page_table.dim() != 2:
            raise ValueError(f"page_table: shape {tuple(self.page_table.shape)}, expected [rows, max_pages]")
        rows, width = self.page_table.shape
        _need(self.page_table, "page_table", torch.int32, (rows, width), dev)
        _need(self.seq_lens, "seq_lens", torch.int32, (rows,), dev)
        _need(self.page_refs, "page_refs", torch.int32, (pages,), dev)
        _need(self.err_word, "err_word", torch.int32, (1,), dev)
        codes = self.k.dtype in _CODES
        if codes:
            for name, t in (("k_scale", self.k_scale), ("v_scale", self.v_scale)):
                if t is None:
                    raise ValueError(f"{name} is required with a {'4-bit' if self.k.dtype == torch.uint8 else 'float8_e4m3fn'} cache")
                _need(t, name, torch.float32, (layers, Hkv), dev)
        st = _Cache(_ptr(self.k), _ptr(self.v), _TYPES[self.k.dtype], layers, pages, Hkv, ps, D, rows, width,
                    _ptr(self.page_table), _ptr(self.seq_lens), _ptr(self.page_refs),
                    _ptr(self.k_scale) if codes else None, _ptr(self.v_scale) if codes else None, _ptr(self.err_word))
        d.pop("_plans", None)
        d["_c_struct"] = cached = (st, ctypes.byref(st), ptrs, dev)
        self._make_workspaces()
        return cached

    def _make_workspaces(self):
        """Makes and clears the cache's own workspaces, where there are none that fit its tensors.  The clear
        (and that of an error word made here) has run when this returns, so that no stream needs an order
        with it.  Inside a capture it would only run with the graph: none is made there."""
        d, dev = self.__dict__, self.k.device
        if self.k.dim() != 5 or self.page_table.dim() != 2:
            return
        capturing = _capturing(dev)
        st = _Cache(num_pages=self.k.shape[1], head_dim=self.head_dim, rows=self.page_table.shape[0])
        made = False
        for kind, size in (("_kv_ws", _lib.kda_kv_workspace_size), ("_attn_ws", _lib.kda_attn_workspace_size)):
            n, old = max(256, int(size(ctypes.byref(st)))), d.get(kind)
            if old is not None and old.numel() >= n and old.device == dev:
                continue
            if capturing:
                d[kind] = None
            else:
                if old is not None and old.is_cuda:
                    torch.cuda.synchronize(old.device)   # calls on any stream may still use it
                d[kind] = torch.zeros(n, dtype=torch.uint8, device=dev)
                made = True
        if made and dev.type == "cuda":
            torch.cuda.current_stream(dev).synchronize()

    def _workspace(self, kind: str, given: Optional[torch.Tensor]) -> Tuple[int, int]:
        """(pointer, bytes) of the given workspace, or of the cache's own."""
        if given is not None:
            if given.device != self.device or not given.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on the cache's device")
            return given.data_ptr(), given.numel() * given.element_size()
        own = self.__dict__.get(kind)
        if own is None:
            self._make_workspaces()
            own = self.__dict__.get(kind)
            if own is None:
                raise RuntimeError("no workspace can be made while a graph is captured: make the cache before the capture, or pass workspace=")
        return own.data_ptr(), own.numel()


def _capturing(dev: torch.device) -> bool:
    """Whether the current stream of this device is being captured into a graph."""
    if dev.type != "cuda":
        return False
    with torch.cuda.device(dev):
        return torch.cuda.is_current_stream_capturing()


def kda_kv_workspace_size(cache: KdaKvCache) -> int:
    return int(_lib.kda_kv_workspace_size(ctypes.byref(cache.c_struct())))


def kda_attn_workspace_size(cache: KdaKvCache) -> int:
    return int(_lib.kda_attn_workspace_size(ctypes.byref(cache.c_struct())))


def _i32(x, name: str) -> int:
    """x as a C int32 (ctypes would cut higher bits off in silence)."""
    x = int(x)
    if not -1 << 31 <= x < 1 << 31:
        raise ValueError(f"{name}={x} does not fit 32 bits")
    return x


def _ints(t: torch.Tensor, name: str, n: int, dev) -> int:
    _need(t, name, torch.int32, (n,), dev)
    return t.data_ptr()


def _rows(t: torch.Tensor, dev, name: str = "rows") -> Tuple[int, int]:
    """(pointer, B) of an int32 [B] tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError(f"{name} must be an int32 tensor [B]")
    n = t.shape[0]
    _need(t, name, torch.int32, (n,), dev)
    return t.data_ptr(), n


def kda_kv_extend(cache: KdaKvCache, rows, n_tokens: Union[int, torch.Tensor], workspace=None, stream=None) -> None:
    """Pages and length for n_tokens (an int, or int32 [B]) more tokens of each row in rows (int32 [B],
    distinct), once per step for all layers; a partly filled last page that others share is copied."""
    _, st, _, dev = cache._struct()
    pr, B = _rows(rows, dev)
    pn, n = (None, _i32(n_tokens, "n_tokens")) if not isinstance(n_tokens, torch.Tensor) else (_ints(n_tokens, "n_tokens", B, dev), 0)
    ws, nb = cache._workspace("_kv_ws", workspace)
    _call(dev, _lib.kda_kv_extend, st, pr, pn, n, B, ws, nb, _stream(stream, dev))


def kda_kv_truncate(cache: KdaKvCache, rows, new_lens, workspace=None, stream=None) -> None:
    """Cuts each row to new_lens (int32 [B]) tokens; 0 frees it.  Drafts that were not accepted."""
    _, st, _, dev = cache._struct()
    pr, B = _rows(rows, dev)
    ws, nb = cache._workspace("_kv_ws", workspace)
    _call(dev, _lib.kda_kv_truncate, st, pr, _ints(new_lens, "new_lens", B, dev), B, ws, nb, _stream(stream, dev))


def kda_kv_fork(cache: KdaKvCache, src_rows, dst_rows, workspace=None, stream=None) -> None:
    """Each dst row gives its pages back and shares all pages of its src row (int32 [n] both)."""
    _, st, _, dev = cache._struct()
    ps, n = _rows(src_rows, dev, "src_rows")
    ws, nb = cache._workspace("_kv_ws", workspace)
    _call(dev, _lib.kda_kv_fork, st, ps, _ints(dst_rows, "dst_rows", n, dev), n, ws, nb, _stream(stream, dev))


def kda_kv_compact(cache: KdaKvCache, remap=None, workspace=None, stream=None) -> torch.Tensor:
    """Moves the pages in use to the lowest ids; returns the new id of each page (int32 [pages], -1:
    free before)."""
    _, st, _, dev = cache._struct()
    if remap is None:
        remap = torch.empty(cache.num_pages, dtype=torch.int32, device=dev)
    ws, nb = cache._workspace("_kv_ws", workspace)
    _call(dev, _lib.kda_kv_compact, st, _ints(remap, "remap", cache.num_pages, dev), ws, nb, _stream(stream, dev))
    return remap


def _tokens(t: torch.Tensor, name: str, packed: bool, heads: Optional[int], cache: KdaKvCache) -> _Layout:
    """Layout of [B, T, heads, D] or, packed, [N, heads, D]: any strides, the last dimension contiguous."""
    D, dev = cache.head_dim, cache.device
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name}: dtype {t.dtype}, expected bfloat16 or float16")
    if cache.k.dtype not in _CODES and cache.k.dtype != t.dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, the cache holds {cache.k.dtype}")
    n = t.shape
    if len(n) != (3 if packed else 4) or n[-1] != D or (heads is not None and n[-2] != heads):
        raise ValueError(f"{name}: shape {tuple(n)}, expected {'[N' if packed else '[B, T'}, "
                         f"{'Hq' if heads is None else heads}, {D}]")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, expected {dev}")
    _i32(max(n), f"{name}: size")
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"{name}: its last dimension must be contiguous")
    # a dimension of one element has no stride to speak of
    return _Layout(_TYPES[t.dtype], 0 if packed or n[0] == 1 else st[0], 0 if n[-3] == 1 else st[-3], 0 if n[-2] == 1 else st[-2])


def _plan(cache: KdaKvCache, key, make):
    """What `make` works out for calls of this form (types, shapes, strides): checked and built at the
    first one, kept with the cache, a few hundred at most."""
    plans = cache.__dict__.get("_plans")
    if plans is None:
        plans = cache.__dict__["_plans"] = {}
    got = plans.get(key)
    if got is None:
        if len(plans) >= 512:
            plans.clear()
        got = plans[key] = make()
    return got


def kda_kv_append(cache: KdaKvCache, layer: int, rows, k, v, cu_seqlens=None, n_tokens=None, stream=None) -> None:
    """Writes the new keys and values of a layer into their pages (after kda_kv_extend).  k, v are
    [B, T, Hkv, D], or packed [N, Hkv, D] with cu_seqlens int32 [B+1]; without it a packed [N, Hkv, D]
    holds N / B tokens of each row.  n_tokens int32 [B]: the first n of the T tokens count."""
    _, st, _, dev = cache._struct()
    pr, B = _rows(rows, dev)
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")

    def make():
        packed = k.dim() == 3
        kl, vl = _tokens(k, "k", packed, cache.Hkv, cache), _tokens(v, "v", packed, cache.Hkv, cache)
        if k.shape != v.shape:
            raise ValueError(f"k and v have shapes {tuple(k.shape)} and {tuple(v.shape)}")
        if cu_seqlens is not None:
            if not packed:
                raise ValueError("cu_seqlens goes with packed k and v [N, Hkv, D]")
            T = k.shape[0]
        elif packed:
            if B and k.shape[0] % B:
                raise ValueError(f"{k.shape[0]} packed tokens are no multiple of {B} rows: pass cu_seqlens")
            T = k.shape[0] // B if B else 0
            kl.seq_stride, vl.seq_stride = T * kl.token_stride, T * vl.token_stride
        else:
            if k.shape[0] != B:
                raise ValueError(f"k: {k.shape[0]} sequences, rows has {B}")
            T = k.shape[1]
        return T, ctypes.byref(kl), ctypes.byref(vl)

    T, kl, vl = _plan(cache, ("append", B, cu_seqlens is None, k.dtype, v.dtype, k.device, v.device, k.shape, v.shape, k.stride(), v.stride()), make)
    pc = None if cu_seqlens is None else _ints(cu_seqlens, "cu_seqlens", B + 1, dev)
    pn = None if n_tokens is None else _ints(n_tokens, "n_tokens", B, dev)
    _call(dev, _lib.kda_kv_append, st, _i32(layer, "layer"), pr, B, T, pn, pc, k.data_ptr(), kl, v.data_ptr(), vl, _stream(stream, dev))


def _attn(cache: KdaKvCache, q, packed: bool, scale, window, sinks, out, lse, return_lse):
    """Descriptor, output and lse of an attention call."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    shape = q.shape
    # plain numbers, so that a plan is found by their values (a tensor would be found by its identity)
    if scale is not None and type(scale) is not float:
        scale = float(scale)
    if type(window) is not int:
        window = int(window)
    if type(sinks) is not int:
        sinks = int(sinks)

    def make():
        ql = _tokens(q, "q", packed, None, cache)
        D = cache.head_dim
        desc = _Desc(shape[-2], 1.0 / math.sqrt(D) if scale is None else scale, _i32(window, "window"), _i32(sinks, "sinks"), ql)
        return ctypes.byref(desc), shape[:-1]

    desc, rows_shape = _plan(cache, ("attn", packed, scale, window, sinks, q.dtype, q.device, shape, q.stride()), make)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _need(out, "out", q.dtype, shape, q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, rows_shape, q.device)
    elif return_lse:
        lse = torch.empty(rows_shape, dtype=torch.float32, device=q.device)
    return desc, out, lse


def kda_attn_decode(cache: KdaKvCache, layer: int, rows, q, scale: Optional[float] = None, window: int = 0,
                    sinks: int = 0, n_tokens=None, out=None, lse=None, return_lse: bool = False, workspace=None,
                    stream=None):
    """Attention of the last T (1..16) tokens of each row over the layer's pages; q [B, T, Hq, D] (strides in
    multiples of 8 elements, the last dimension contiguous).  A workspace that is passed has to be zeroed once by its owner.
    Causal, or with a sliding window and sinks first tokens that stay visible.  n_tokens int32 [B]: only
    the first n of the T tokens count (entries past them are left as they were).  Returns out, or
    (out, lse f32 [B, T, Hq]) where lse is given or return_lse is set."""
    _, st, _, dev = cache._struct()
    pr, B = _rows(rows, dev)
    desc, out, lse = _attn(cache, q, False, scale, window, sinks, out, lse, return_lse)
    if q.shape[0] != B:
        raise ValueError(f"q: {q.shape[0]} sequences, rows has {B}")
    pn = None if n_tokens is None else _ints(n_tokens, "n_tokens", B, dev)
    ws, nb = cache._workspace("_attn_ws", workspace)
    _call(dev, _lib.kda_attn_decode, st, _i32(layer, "layer"), desc, pr, B, q.shape[1], pn, q.data_ptr(), out.data_ptr(), _ptr(lse), ws, nb,
          _stream(stream, dev))
    return out if lse is None else (out, lse)


def kda_attn_prefill(cache: KdaKvCache, layer: int, rows, cu_seqlens, max_len: int, q, scale: Optional[float] = None,
                     window: int = 0, sinks: int = 0, out=None, lse=None, return_lse: bool = False, workspace=None,
                     stream=None):
    """Attention of packed new tokens: sequence b is rows cu_seqlens[b]..cu_seqlens[b+1]-1 of q [N, Hq, D],
    the last tokens of cache row rows[b]; max_len bounds every count (host int, no device read).  q may have any
    strides in multiples of 8 elements, its last dimension contiguous; a workspace that is passed has to be zeroed once by its owner.
    Returns out, or (out, lse f32 [N, Hq]) where lse is given or return_lse is set."""
    _, st, _, dev = cache._struct()
    pr, B = _rows(rows, dev)
    desc, out, lse = _attn(cache, q, True, scale, window, sinks, out, lse, return_lse)
    pc = _ints(cu_seqlens, "cu_seqlens", B + 1, dev)
    ws, nb = cache._workspace("_attn_ws", workspace)
    _call(dev, _lib.kda_attn_prefill, st, _i32(layer, "layer"), desc, pr, B, pc, q.shape[0], _i32(max_len, "max_len"), q.data_ptr(), out.data_ptr(), _ptr(lse),
          ws, nb, _stream(stream, dev))
    return out if lse is None else (out, lse)


def kda_kv_get_error(cache: KdaKvCache, stream=None) -> int:
    """Reads and clears the cache's device error word (synchronises the stream).  After KDA_DEVERR_TIMEOUT the
    cache's own attention workspace is cleared as well; one that was passed has to be cleared by its owner."""
    _, st, _, dev = cache._struct()
    v = ctypes.c_int32(0)
    with torch.cuda.device(dev):
        r = _lib.kda_kv_get_error(st, ctypes.byref(v), _stream(stream, dev))
    if r not in (KDA_OK, KDA_ERR_DEVICE):
        _raise(r)
    own = cache.__dict__.get("_attn_ws")
    if v.value & KDA_DEVERR_TIMEOUT and own is not None:
        own.zero_()
        if own.is_cuda:
            torch.cuda.current_stream(dev).synchronize()
    return int(v.value)
