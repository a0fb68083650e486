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
_SCALE = 1.0 / math.sqrt(128)

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
_bf16, _f16, _f32_t, _i32_t = torch.bfloat16, torch.float16, torch.float32, torch.int32
_D = 128


# These calls are used once per layer and token, so the checks below avoid
# everything that costs a microsecond on the host: no torch.device objects, no
# per-call list conversions, no import statements.
_fns: dict = {}


def _fn(name: str):
    f = _fns.get(name)
    if f is None:
        import long_context_hybrid_b200 as base
        f = _fns[name] = getattr(base.lib(), name)
    return f


def _refuse(what: str):
    import long_context_hybrid_b200 as base
    raise base.RtpError(what)


def _device(what: str, *tensors) -> int:
    """Index of the one CUDA device that every tensor (None skipped) is on."""
    dev = tensors[0].get_device()
    if dev < 0:
        _refuse(f"{what}: CUDA tensors only")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _refuse(f"{what}: tensors on different devices")
    return dev


def _int32(what: str, t: torch.Tensor, n: int) -> int:
    if t.dtype is not _i32_t or t.shape != (n,) or not t.is_contiguous():
        _refuse(f"{what}: a contiguous int32 vector of {n}")
    return t.data_ptr()


def _rows(what: str, t: torch.Tensor, shape, dtype) -> Strides:
    if t.dtype is not dtype or t.shape != shape:
        _refuse(f"{what}: expected {dtype} {tuple(shape)}")
    n, h, d = t.stride()
    if d != 1:
        _refuse(f"{what}: the last dimension must be contiguous")
    return Strides(0, n, h)


def _f32(what: str, t: torch.Tensor, shape) -> int:
    if t.dtype is not _f32_t or t.shape != shape or not t.is_contiguous():
        _refuse(f"{what}: expected contiguous float32 {tuple(shape)}")
    return t.data_ptr()


def _bounds(cu: torch.Tensor) -> int:
    if cu.dim() != 1 or cu.shape[0] < 2:
        _refuse("cu_seqlens: an int32 vector of at least two bounds")
    return cu.shape[0] - 1


@functools.lru_cache(maxsize=256)
def _head_array(heads: tuple):
    return (ctypes.c_int32 * len(heads))(*[int(h) for h in heads])


def _stream(dev: int, stream) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, dev: int, stream) -> torch.Tensor:
    """Scratch that belongs to the stream it is used on, so that its memory is not handed out before the work ends."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _workspace(nbytes: int, dev: int, ws: Optional[torch.Tensor], stream) -> torch.Tensor:
    if ws is None:
        return _empty(nbytes, torch.uint8, dev, stream)
    if ws.get_device() != dev or not ws.is_contiguous():
        _refuse("ws: a contiguous tensor on the call's device")
    return ws


def _run(name: str, dev: int, *args) -> None:
    """The C call with its tensors' device current."""
    if dev == torch._C._cuda_getDevice():
        status = _fn(name)(*args)
    else:
        with torch.cuda.device(dev):
            status = _fn(name)(*args)
    if status != 0:
        import long_context_hybrid_b200 as base
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
        shape, dtype = k.shape, k.dtype
        if len(shape) != 4 or dtype not in _DTYPES or v.shape != shape or v.dtype is not dtype or shape[3] != _D:
            _refuse(f"PagedCache: k and v [num_pages, page_size, Hkv, {_D}], bf16 or fp16 alike")
        kp, kn, kh, kd = k.stride()
        vp, vn, vh, vd = v.stride()
        if kd != 1 or vd != 1:
            _refuse("PagedCache: D must be contiguous")
        if table.dtype is not _i32_t or table.dim() != 2:
            _refuse("PagedCache: table int32 [B, max_pages]")
        B, n = table.shape
        row, step = table.stride()
        if n > 1 and step != 1:
            _refuse("PagedCache: the table's rows must be contiguous")
        self.dev = _device("PagedCache", k, v, table, weights)
        P, page, Hkv, _ = shape
        w = None if weights is None else _f32("PagedCache: weights", weights, (P, Hkv, page))
        self.k, self.v, self.table, self.weights = k, v, table, weights
        self.num_pages, self.page_size, self.Hkv, self.D, self.dtype = P, page, Hkv, _D, dtype
        self.B, self.capacity = B, n * page
        self.struct = _CacheStruct(k.data_ptr(), v.data_ptr(), Strides(kp, kn, kh), Strides(vp, vn, vh), w,
                                   table.data_ptr(), row if B > 1 else max(n, 1), P, page, n, Hkv)


def attn_packed(q, k, v, o, heads: Sequence[int], cu_seqlens, window: Optional[int] = None,
                scale: Optional[float] = None, lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                stream=None):
    """Causal attention of packed prompts: q/o [T,Hq,D], k/v [T,Hkv,D],
    ``cu_seqlens`` int32 [S+1] on the device; writes o[:, heads] (rows of
    sequences) and ``lse`` fp32 [len(heads), T]. ``window`` None: the whole
    prefix."""
    T, Hq, D = shape = q.shape
    kshape, dtype = k.shape, q.dtype
    dev = _device("attn_packed", q, k, v, o, cu_seqlens, lse)
    if dtype not in _DTYPES or D != _D or len(kshape) != 3 or kshape[0] != T or kshape[2] != D:
        _refuse("attn_packed: q [T, Hq, 128] and k [T, Hkv, 128], bf16 or fp16")
    S = _bounds(cu_seqlens)
    heads = _head_array(tuple(heads))
    n = len(heads)
    buf = _workspace(256, dev, ws, stream)
    _run("rtp_attn_packed", dev, q.data_ptr(), _rows("q", q, shape, dtype), k.data_ptr(),
         _rows("k", k, kshape, dtype), v.data_ptr(), _rows("v", v, kshape, dtype), o.data_ptr(),
         _rows("o", o, shape, dtype), _DTYPES[dtype], T, Hq, kshape[1], heads, n,
         _int32("cu_seqlens", cu_seqlens, S + 1), S, _INT32_MAX if window is None else window,
         _SCALE if scale is None else scale, None if lse is None else _f32("lse", lse, (n, T)), buf.data_ptr(),
         buf.nbytes, _stream(dev, stream))
    return o


def attn_key_weights(q, k, lse, weights, heads: Sequence[int], cu_seqlens, n_obs: Optional[int] = None,
                     window: Optional[int] = None, scale: Optional[float] = None, ws: Optional[torch.Tensor] = None,
                     stream=None):
    """The attention weight each key of packed prompts got from the last
    ``n_obs`` rows of its sequence (None: every row), summed over the listed
    heads of its KV head, into ``weights`` fp32 [Hkv, T]; ``lse`` fp32
    [len(heads), T] from ``attn_packed``."""
    T, Hq, D = shape = q.shape
    kshape, dtype = k.shape, q.dtype
    dev = _device("attn_key_weights", q, k, lse, weights, cu_seqlens)
    if dtype not in _DTYPES or D != _D or len(kshape) != 3 or kshape[0] != T or kshape[2] != D:
        _refuse("attn_key_weights: q [T, Hq, 128] and k [T, Hkv, 128], bf16 or fp16")
    S = _bounds(cu_seqlens)
    heads = _head_array(tuple(heads))
    n = len(heads)
    buf = _workspace(256, dev, ws, stream)
    _run("rtp_attn_key_weights", dev, q.data_ptr(), _rows("q", q, shape, dtype), k.data_ptr(),
         _rows("k", k, kshape, dtype), _DTYPES[dtype], T, Hq, kshape[1], heads, n,
         _int32("cu_seqlens", cu_seqlens, S + 1), S, _f32("lse", lse, (n, T)), _INT32_MAX if n_obs is None else n_obs,
         _INT32_MAX if window is None else window, _SCALE if scale is None else scale,
         _f32("weights", weights, (kshape[1], T)), buf.data_ptr(), buf.nbytes, _stream(dev, stream))
    return weights


def paged_append(cache: PagedCache, k, v, cu_seqlens, pos, weights: Optional[torch.Tensor] = None, stream=None):
    """Puts new tokens into the cache: row t of sequence i (k/v [T,Hkv,D],
    ``cu_seqlens`` int32 [S+1]) goes to slot pos[i] + t - cu_seqlens[i] of
    table row i. ``weights`` fp32 [Hkv,T] starts their accumulated weights
    (None: 0)."""
    T = k.shape[0]
    shape, dtype = (T, cache.Hkv, _D), cache.dtype
    dev = _device("paged_append", cache.k, k, v, cu_seqlens, pos, weights)
    S = _bounds(cu_seqlens)
    if S > cache.B:
        _refuse("paged_append: more sequences than table rows")
    _run("rtp_paged_append", dev, cache.struct, k.data_ptr(), _rows("k", k, shape, dtype), v.data_ptr(),
         _rows("v", v, shape, dtype), None if weights is None else _f32("weights", weights, (cache.Hkv, T)), T,
         _int32("cu_seqlens", cu_seqlens, S + 1), S, _int32("pos", pos, S), _stream(dev, stream))


def paged_attn_decode(q, cache: PagedCache, lens, o, heads: Sequence[int], window: Optional[int] = None,
                      sink: int = 0, scale: Optional[float] = None, max_len: Optional[int] = None,
                      lse: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None):
    """One new token per sequence over the paged cache: q/o [B,Hq,D], ``lens``
    int32 [B]; attends the slots [0, sink) and the last ``window`` (None: all).
    ``max_len`` (default: the table's capacity) bounds the lengths. ``lse``
    fp32 [B,len(heads)]; ``weights_out`` (like cache.weights, may be it)
    receives cache.weights plus this token's attention weights."""
    B, Hq, _ = q.shape
    shape, dtype = (B, Hq, _D), cache.dtype
    dev = _device("paged_attn_decode", cache.k, q, lens, o, lse, weights_out)
    qs, os_ = _rows("q", q, shape, dtype), _rows("o", o, shape, dtype)
    qs.b, os_.b = qs.n, os_.n
    if B > cache.B:
        _refuse("paged_attn_decode: more sequences than table rows")
    heads = _head_array(tuple(heads))
    n = len(heads)
    if max_len is None:
        max_len = cache.capacity
    if window is None:
        window = _INT32_MAX
    w = None
    if weights_out is not None:
        w = _f32("weights_out", weights_out, (cache.num_pages, cache.Hkv, cache.page_size))
    buf = _workspace(_fn("rtp_workspace_size_paged_attn_decode")(B, max_len, n, window, sink, w is not None), dev, ws,
                     stream)
    _run("rtp_paged_attn_decode", dev, q.data_ptr(), qs, cache.struct, _int32("lens", lens, B), max_len, o.data_ptr(),
         os_, _DTYPES[dtype], B, Hq, heads, n, window, sink, _SCALE if scale is None else scale,
         None if lse is None else _f32("lse", lse, (B, n)), w, buf.data_ptr(), buf.nbytes, _stream(dev, stream))
    return o


def cache_evict(cache: PagedCache, lens, budget: int, sink: int = 0, recent: int = 0,
                out: Optional[PagedCache] = None, idx: Optional[torch.Tensor] = None,
                new_lens: Optional[torch.Tensor] = None, max_len: Optional[int] = None, stream=None):
    """Shrinks the cache to ``budget`` tokens per sequence and KV head: the
    first ``sink``, the last ``recent`` and the others of largest accumulated
    weight, moved to slots 0, 1, ... of ``out`` (default: in place). Returns
    (idx int32 [B,Hkv,budget], the kept slots ascending and -1 padded; new_lens
    int32 [B])."""
    if out is None:
        out = cache
    B = lens.shape[0]
    dev = _device("cache_evict", cache.k, lens, out.k, idx, new_lens)
    if cache.dtype is not out.dtype:
        _refuse("cache_evict: caches of different types")
    if cache.weights is None or out.weights is None:
        _refuse("cache_evict: both caches need weights")
    if B > cache.B or B > out.B:
        _refuse("cache_evict: more sequences than table rows")
    if idx is None:
        idx = _empty((B, cache.Hkv, budget), _i32_t, dev, stream)
    if new_lens is None:
        new_lens = _empty((B,), _i32_t, dev, stream)
    if idx.dtype is not _i32_t or idx.shape != (B, cache.Hkv, budget) or not idx.is_contiguous():
        _refuse(f"idx: expected contiguous int32 {(B, cache.Hkv, budget)}")
    _run("rtp_cache_evict", dev, cache.struct, out.struct, B, _int32("lens", lens, B),
         cache.capacity if max_len is None else max_len, budget, sink, recent, idx.data_ptr(),
         _int32("new_lens", new_lens, B), _stream(dev, stream))
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
        if self.streaming and window is None:
            _refuse("PagedLayer: streaming heads need a window")
        self.scale = scale
        B, dev = cache.B, cache.dev
        self.lens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.cu_decode = torch.arange(B + 1, dtype=torch.int32, device=dev)
        self.ws_prefill = torch.zeros(256, dtype=torch.uint8, device=dev)
        weighed = cache.weights is not None
        size = _fn("rtp_workspace_size_paged_attn_decode")
        self.ws = torch.empty(max(size(B, cache.capacity, max(1, len(g)), _INT32_MAX if w is None else w, sink, weighed)
                                  for g, w in self._groups()), dtype=torch.uint8, device=dev)

    def _groups(self):
        """(heads, window) of the two kinds of heads that are there."""
        return [x for x in ((self.full, None), (self.streaming, self.window)) if x[0]]

    def prefill(self, q, k, v, o, cu_seqlens, stream=None):
        """q/o [T,Hq,D], k/v [T,Hkv,D] of B packed prompts (one per table row)."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.cache.dev)):
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
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.cache.dev)):
            paged_append(self.cache, k, v, self.cu_decode, self.lens)
            self.lens.add_(1)
            for heads, window in self._groups():
                paged_attn_decode(q, self.cache, self.lens, o, heads, window, self.sink if window else 0, self.scale,
                                  weights_out=self.cache.weights, ws=self.ws)
        return o

    def evict(self, budget: int, recent: int, stream=None):
        """Shrinks every sequence to ``budget`` tokens per KV head, keeping the
        ``sink`` first and ``recent`` last; returns the kept slots."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.cache.dev)):
            idx, new_lens = cache_evict(self.cache, self.lens, budget, self.sink, recent)
            self.lens.copy_(new_lens)
        return idx
