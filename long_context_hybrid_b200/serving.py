"""Serving calls: packed prompts, a paged key-value cache and its eviction.

Marshalling for the serving part of ``include/rtp.h`` and ``PagedLayer``,
which runs the calls of one layer in order. Arguments that the C side cannot
see (dtypes, shapes, devices, contiguity) are checked here and raise
``RtpError``; the rest is checked by the C calls. Work goes to the current
stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Sequence

import torch

_INT32_MAX = 2**31 - 1


def _base():
    import long_context_hybrid_b200 as base
    return base


class Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("n", ctypes.c_int64), ("h", ctypes.c_int64)]


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", Strides), ("vs", Strides),
                ("weights", ctypes.c_void_p), ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("Hkv", ctypes.c_int32)]


_P, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_H = ctypes.POINTER(ctypes.c_int32)
_C = ctypes.POINTER(_CacheStruct)

SIGNATURES = {
    "rtp_workspace_size_attn_packed": (_SZ, []),
    "rtp_attn_packed": (_I, [_P, Strides, _P, Strides, _P, Strides, _P, Strides, _I, _I, _I, _I, _H, _I, _P, _I, _I, _F,
                             _P, _P, _SZ, _P]),
    "rtp_workspace_size_attn_key_weights": (_SZ, []),
    "rtp_attn_key_weights": (_I, [_P, Strides, _P, Strides, _I, _I, _I, _I, _H, _I, _P, _I, _P, _I, _I, _F, _P, _P, _SZ,
                                  _P]),
    "rtp_paged_append": (_I, [_C, _P, Strides, _P, Strides, _P, _I, _P, _I, _P, _P]),
    "rtp_workspace_size_paged_attn_decode": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "rtp_paged_attn_decode": (_I, [_P, Strides, _C, _P, _I, _P, Strides, _I, _I, _I, _H, _I, _I, _I, _F, _P, _P, _P, _SZ,
                                   _P]),
    "rtp_cache_evict": (_I, [_C, _C, _I, _P, _I, _I, _I, _I, _P, _P, _P]),
}

_DTYPES = {torch.bfloat16: 0, torch.float16: 2}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise _base().RtpError(what)


def _same_device(what: str, first: torch.Tensor, *others) -> torch.device:
    dev = first.device
    _need(dev.type == "cuda", f"{what}: CUDA tensors only")
    for t in others:
        _need(t is None or t.device == dev, f"{what}: tensors on different devices")
    return dev


def _int32(what: str, t: torch.Tensor, n: Optional[int] = None) -> int:
    _need(t.dtype == torch.int32 and t.dim() == 1 and t.is_contiguous() and (n is None or t.shape[0] == n),
          f"{what}: a contiguous int32 vector" + ("" if n is None else f" of {n}"))
    return t.data_ptr()


def _rows(what: str, t: torch.Tensor, shape, dtype) -> Strides:
    _need(t.dtype == dtype and tuple(t.shape) == tuple(shape), f"{what}: expected {dtype} {tuple(shape)}")
    _need(t.stride(-1) == 1, f"{what}: the last dimension must be contiguous")
    return Strides(0, t.stride(0), t.stride(1))


def _f32(what: str, t: torch.Tensor, shape) -> int:
    _need(t.dtype == torch.float32 and tuple(t.shape) == tuple(shape) and t.is_contiguous(),
          f"{what}: expected contiguous float32 {tuple(shape)}")
    return t.data_ptr()


@functools.lru_cache(maxsize=256)
def _head_array(heads: tuple):
    return (ctypes.c_int32 * len(heads))(*heads)


def _heads(heads: Sequence[int]):
    h = tuple(int(x) for x in heads)
    return _head_array(h), len(h)


def _scale(scale: Optional[float], D: int) -> float:
    return 1.0 / math.sqrt(D) if scale is None else scale


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Scratch that belongs to the stream it is used on, so that its memory is not handed out before the work ends."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(nbytes: int, device, ws: Optional[torch.Tensor], stream) -> torch.Tensor:
    if ws is None:
        return _empty(nbytes, torch.uint8, device, stream)
    _need(ws.device == device and ws.is_contiguous(), "ws: a contiguous tensor on the call's device")
    return ws


def _run(name: str, dev: torch.device, stream, *args) -> None:
    """The C call on `stream` (default: the device's current one), with that device current."""
    base = _base()
    fn = getattr(base.lib(), name)
    if dev.index == torch.cuda.current_device():
        status = fn(*args, (stream or torch.cuda.current_stream()).cuda_stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, (stream or torch.cuda.current_stream(dev)).cuda_stream)
    base._check(status, name)


class PagedCache:
    """A paged key-value cache: ``k``, ``v`` [num_pages, page_size, Hkv, D]
    (bf16 or fp16; any strides with contiguous D, so a head-major pool works as
    a transposed view), ``table`` int32 [B, max_pages] with contiguous rows, and
    optionally ``weights`` fp32 [num_pages, Hkv, page_size], the accumulated
    attention weight of every cached token. Slot s of sequence b is row
    s % page_size of page table[b, s // page_size]. The tensors are the
    caller's; the pages they hold are written by ``paged_append`` and
    ``cache_evict``."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, weights: Optional[torch.Tensor] = None):
        _need(k.dim() == 4 and k.dtype in _DTYPES and v.shape == k.shape and v.dtype == k.dtype,
              "PagedCache: k and v [num_pages, page_size, Hkv, D], bf16 or fp16 alike")
        P, page, Hkv, D = k.shape
        _need(D == _base().D_HEAD, f"PagedCache: D must be {_base().D_HEAD}")
        _need(k.stride(3) == 1 and v.stride(3) == 1, "PagedCache: D must be contiguous")
        _need(table.dim() == 2 and table.dtype == torch.int32 and (table.shape[1] <= 1 or table.stride(1) == 1),
              "PagedCache: table int32 [B, max_pages] with contiguous rows")
        self.device = _same_device("PagedCache", k, v, table, weights)
        w = None if weights is None else _f32("PagedCache: weights", weights, (P, Hkv, page))
        self.k, self.v, self.table, self.weights = k, v, table, weights
        self.num_pages, self.page_size, self.Hkv, self.D = P, page, Hkv, D
        B, n = table.shape
        self.struct = _CacheStruct(k.data_ptr(), v.data_ptr(), Strides(k.stride(0), k.stride(1), k.stride(2)),
                                   Strides(v.stride(0), v.stride(1), v.stride(2)), w, table.data_ptr(),
                                   table.stride(0) if B > 1 else max(n, 1), P, page, n, Hkv)

    @property
    def capacity(self) -> int:
        return self.table.shape[1] * self.page_size


def attn_packed(q, k, v, o, heads: Sequence[int], cu_seqlens, window: Optional[int] = None,
                scale: Optional[float] = None, lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                stream=None):
    """Causal attention of packed prompts: q/o [T,Hq,D], k/v [T,Hkv,D],
    ``cu_seqlens`` int32 [S+1] on the device; writes o[:, heads] (rows of
    sequences) and ``lse`` fp32 [len(heads), T]. ``window`` None: the whole
    prefix."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    dev = _same_device("attn_packed", q, k, v, o, cu_seqlens, lse)
    _need(q.dtype in _DTYPES and D == _base().D_HEAD, "attn_packed: bf16 or fp16, D = 128")
    qs, ks = _rows("q", q, (T, Hq, D), q.dtype), _rows("k", k, (T, Hkv, D), q.dtype)
    vs, os_ = _rows("v", v, (T, Hkv, D), q.dtype), _rows("o", o, (T, Hq, D), q.dtype)
    h, n_heads = _heads(heads)
    lse_p = None if lse is None else _f32("lse", lse, (n_heads, T))
    buf = _workspace(256, dev, ws, stream)
    _run("rtp_attn_packed", dev, stream, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, o.data_ptr(), os_,
         _DTYPES[q.dtype], T, Hq, Hkv, h, n_heads, _int32("cu_seqlens", cu_seqlens), cu_seqlens.shape[0] - 1,
         _INT32_MAX if window is None else window, _scale(scale, D), lse_p, buf.data_ptr(), buf.nbytes)
    return o


def attn_key_weights(q, k, lse, weights, heads: Sequence[int], cu_seqlens, n_obs: Optional[int] = None,
                     window: Optional[int] = None, scale: Optional[float] = None, ws: Optional[torch.Tensor] = None,
                     stream=None):
    """The attention weight each key of packed prompts got from the last
    ``n_obs`` rows of its sequence (None: every row), summed over the listed
    heads of its KV head, into ``weights`` fp32 [Hkv, T]; ``lse`` fp32
    [len(heads), T] from ``attn_packed``."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    dev = _same_device("attn_key_weights", q, k, lse, weights, cu_seqlens)
    _need(q.dtype in _DTYPES and D == _base().D_HEAD, "attn_key_weights: bf16 or fp16, D = 128")
    qs, ks = _rows("q", q, (T, Hq, D), q.dtype), _rows("k", k, (T, Hkv, D), q.dtype)
    h, n_heads = _heads(heads)
    lse_p, w_p = _f32("lse", lse, (n_heads, T)), _f32("weights", weights, (Hkv, T))
    buf = _workspace(256, dev, ws, stream)
    _run("rtp_attn_key_weights", dev, stream, q.data_ptr(), qs, k.data_ptr(), ks, _DTYPES[q.dtype], T, Hq, Hkv, h,
         n_heads, _int32("cu_seqlens", cu_seqlens), cu_seqlens.shape[0] - 1, lse_p,
         _INT32_MAX if n_obs is None else n_obs, _INT32_MAX if window is None else window, _scale(scale, D), w_p,
         buf.data_ptr(), buf.nbytes)
    return weights


def paged_append(cache: PagedCache, k, v, cu_seqlens, pos, weights: Optional[torch.Tensor] = None, stream=None):
    """Puts new tokens into the cache: row t of sequence i (k/v [T,Hkv,D],
    ``cu_seqlens`` int32 [S+1]) goes to slot pos[i] + t - cu_seqlens[i] of
    table row i. ``weights`` fp32 [Hkv,T] starts their accumulated weights
    (None: 0)."""
    T, Hkv, D = k.shape
    dev = _same_device("paged_append", cache.k, k, v, cu_seqlens, pos, weights)
    _need(Hkv == cache.Hkv, "paged_append: k has another number of KV heads than the cache")
    dtype = cache.k.dtype
    ks, vs = _rows("k", k, (T, Hkv, cache.D), dtype), _rows("v", v, (T, Hkv, cache.D), dtype)
    S = cu_seqlens.shape[0] - 1
    _need(S <= cache.table.shape[0], "paged_append: more sequences than table rows")
    w_p = None if weights is None else _f32("weights", weights, (Hkv, T))
    _run("rtp_paged_append", dev, stream, cache.struct, k.data_ptr(), ks, v.data_ptr(), vs, w_p, T,
         _int32("cu_seqlens", cu_seqlens), S, _int32("pos", pos, S))


def paged_attn_decode(q, cache: PagedCache, lens, o, heads: Sequence[int], window: Optional[int] = None,
                      sink: int = 0, scale: Optional[float] = None, max_len: Optional[int] = None,
                      lse: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None):
    """One new token per sequence over the paged cache: q/o [B,Hq,D], ``lens``
    int32 [B]; attends the slots [0, sink) and the last ``window`` (None: all).
    ``max_len`` (default: the table's capacity) bounds the lengths. ``lse``
    fp32 [B,len(heads)]; ``weights_out`` (like cache.weights, may be it)
    receives cache.weights plus this token's attention weights."""
    B, Hq, D = q.shape
    dev = _same_device("paged_attn_decode", cache.k, q, lens, o, lse, weights_out)
    dtype = cache.k.dtype
    qs, os_ = _rows("q", q, (B, Hq, cache.D), dtype), _rows("o", o, (B, Hq, cache.D), dtype)
    qs, os_ = Strides(qs.n, 0, qs.h), Strides(os_.n, 0, os_.h)
    _need(B <= cache.table.shape[0], "paged_attn_decode: more sequences than table rows")
    h, n_heads = _heads(heads)
    max_len = cache.capacity if max_len is None else max_len
    window = _INT32_MAX if window is None else window
    lse_p = None if lse is None else _f32("lse", lse, (B, n_heads))
    w_p = None
    if weights_out is not None:
        w_p = _f32("weights_out", weights_out, (cache.num_pages, cache.Hkv, cache.page_size))
    need = _base().lib().rtp_workspace_size_paged_attn_decode(B, max_len, n_heads, window, sink, w_p is not None)
    buf = _workspace(need, dev, ws, stream)
    _run("rtp_paged_attn_decode", dev, stream, q.data_ptr(), qs, cache.struct, _int32("lens", lens, B), max_len,
         o.data_ptr(), os_, _DTYPES[dtype], B, Hq, h, n_heads, window, sink, _scale(scale, D), lse_p, w_p,
         buf.data_ptr(), buf.nbytes)
    return o


def cache_evict(cache: PagedCache, lens, budget: int, sink: int = 0, recent: int = 0,
                out: Optional[PagedCache] = None, idx: Optional[torch.Tensor] = None,
                new_lens: Optional[torch.Tensor] = None, max_len: Optional[int] = None, stream=None):
    """Shrinks the cache to ``budget`` tokens per sequence and KV head: the
    first ``sink``, the last ``recent`` and the others of largest accumulated
    weight, moved to slots 0, 1, ... of ``out`` (default: in place). Returns
    (idx int32 [B,Hkv,budget], the kept slots ascending and -1 padded; new_lens
    int32 [B])."""
    out = cache if out is None else out
    B = lens.shape[0]
    dev = _same_device("cache_evict", cache.k, lens, out.k, idx, new_lens)
    _need(cache.k.dtype == out.k.dtype, "cache_evict: caches of different types")
    _need(cache.weights is not None and out.weights is not None, "cache_evict: both caches need weights")
    _need(B <= cache.table.shape[0] and B <= out.table.shape[0], "cache_evict: more sequences than table rows")
    if idx is None:
        idx = _empty((B, cache.Hkv, budget), torch.int32, dev, stream)
    if new_lens is None:
        new_lens = _empty((B,), torch.int32, dev, stream)
    _need(idx.dtype == torch.int32 and tuple(idx.shape) == (B, cache.Hkv, budget) and idx.is_contiguous(),
          f"idx: expected contiguous int32 {(B, cache.Hkv, budget)}")
    max_len = cache.capacity if max_len is None else max_len
    _run("rtp_cache_evict", dev, stream, cache.struct, out.struct, B, _int32("lens", lens, B), max_len, budget, sink,
         recent, idx.data_ptr(), _int32("new_lens", new_lens, B))
    return idx, new_lens


class PagedLayer:
    """One attention layer over a paged cache: prompts, single tokens, eviction.

    ``heads`` attend everything; with ``window`` the ``streaming`` heads attend
    the last ``window`` tokens and, when decoding, the first ``sink``.
    ``prefill`` runs packed prompts and puts their keys and values (and, if the
    cache has weights, the weights that their last ``n_obs`` queries gave) into
    the cache; ``decode`` appends one token per sequence and attends;
    ``evict`` shrinks the cache in place. ``lens`` is the device's record of
    the sequences' lengths, kept by these calls; buffers are kept across calls.
    """

    def __init__(self, cache: PagedCache, Hq: int, streaming: Sequence[int] = (), window: Optional[int] = None,
                 sink: int = 0, n_obs: Optional[int] = None, scale: Optional[float] = None):
        self.cache, self.Hq, self.n_obs, self.window, self.sink = cache, Hq, n_obs, window, sink
        self.streaming = list(streaming)
        self.full = [h for h in range(Hq) if h not in set(self.streaming)]
        _need(not self.streaming or window is not None, "PagedLayer: streaming heads need a window")
        self.scale = _scale(scale, cache.D)
        B, dev = cache.table.shape[0], cache.device
        self.B = B
        self.lens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.cu_decode = torch.arange(B + 1, dtype=torch.int32, device=dev)
        self.ws_prefill = torch.zeros(256, dtype=torch.uint8, device=dev)
        weighed = cache.weights is not None
        size = _base().lib().rtp_workspace_size_paged_attn_decode
        self.ws = torch.empty(max(size(B, cache.capacity, max(1, len(g)), _INT32_MAX if w is None else w, sink, weighed)
                                  for g, w in self._groups()), dtype=torch.uint8, device=dev)

    def _groups(self):
        """(heads, window) of the two kinds of heads that are there."""
        return [x for x in ((self.full, None), (self.streaming, self.window)) if x[0]]

    def prefill(self, q, k, v, o, cu_seqlens, stream=None):
        """q/o [T,Hq,D], k/v [T,Hkv,D] of B packed prompts (one per table row)."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.cache.device)):
            weights = None
            for heads, window in self._groups():
                lse = None
                if self.cache.weights is not None:
                    lse = torch.empty(len(heads), q.shape[0], dtype=torch.float32, device=q.device)
                attn_packed(q, k, v, o, heads, cu_seqlens, window, self.scale, lse, self.ws_prefill)
                if lse is not None:
                    w = torch.zeros(k.shape[1], k.shape[0], dtype=torch.float32, device=q.device)
                    attn_key_weights(q, k, lse, w, heads, cu_seqlens, self.n_obs, window, self.scale,
                                     self.ws_prefill)
                    weights = w if weights is None else weights.add_(w)
            self.lens.zero_()
            paged_append(self.cache, k, v, cu_seqlens, self.lens, weights)
            torch.sub(cu_seqlens[1:], cu_seqlens[:-1], out=self.lens)
        return o

    def decode(self, q, k, v, o, stream=None):
        """q/o [B,Hq,D], k/v [B,Hkv,D]: one new token of every sequence."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.cache.device)):
            paged_append(self.cache, k, v, self.cu_decode, self.lens)
            self.lens.add_(1)
            for heads, window in self._groups():
                paged_attn_decode(q, self.cache, self.lens, o, heads, window, self.sink if window else 0, self.scale,
                                  weights_out=self.cache.weights, ws=self.ws)
        return o

    def evict(self, budget: int, recent: int, stream=None):
        """Shrinks every sequence to ``budget`` tokens per KV head, keeping the
        ``sink`` first and ``recent`` last; returns the kept slots."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.cache.device)):
            idx, new_lens = cache_evict(self.cache, self.lens, budget, self.sink, recent)
            self.lens.copy_(new_lens)
        return idx
