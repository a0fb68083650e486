"""Serving calls: packed prompts, a paged key-value cache and its eviction.

The serving part of ``include/rtp.h`` on torch tensors, and ``PagedLayer``,
which runs the calls of one layer in order. The native module ``_marshal``
reads the tensors; what the C side cannot see (dtypes, shapes, devices,
contiguity) it checks and refuses with ``RtpError``, the rest is checked by the
C calls. Work goes to the given stream, or the current one of the tensors'
device.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Sequence

import torch

_INT32_MAX = 2**31 - 1

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

_native = None


def _marshal():
    """The ``_marshal`` module, set up with the library's functions (raises if either has not been built)."""
    global _native
    if _native is None:
        import long_context_hybrid_b200 as base
        lib = base.lib()
        try:
            from . import _marshal as module
        except ImportError as e:
            raise base.RtpError("_marshal.so is missing: build it with "
                                "`python -m long_context_hybrid_b200.build`") from e

        def address(name):
            return ctypes.cast(getattr(lib, name), ctypes.c_void_p).value

        module.setup(base.RtpError, base._check, torch.bfloat16, torch.float16, torch.float32, torch.int32,
                     torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice, address("rtp_attn_packed"),
                     address("rtp_attn_key_weights"), address("rtp_paged_append"), address("rtp_paged_attn_decode"),
                     address("rtp_cache_evict"), address("rtp_workspace_size_paged_attn_decode"))
        _native = module
    return _native


def _call(name: str, device_of: torch.Tensor, *args) -> None:
    """The native call; it declines where another device than its tensors' is current."""
    f = getattr(_native or _marshal(), name)
    if not f(*args):
        with torch.cuda.device(device_of.get_device()):
            f(*args)


@functools.lru_cache(maxsize=256)
def _head_bytes(heads: tuple) -> bytes:
    return struct.pack(f"{len(heads)}i", *[int(h) for h in heads])


def _empty(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """Scratch that belongs to the stream it is used on, so that its memory is not handed out before the work ends."""
    dev = like.get_device()
    if dev < 0:
        import long_context_hybrid_b200 as base
        raise base.RtpError("CUDA tensors only")
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _bytes(ws: torch.Tensor) -> torch.Tensor:
    return ws if ws.dtype is torch.uint8 else ws.view(torch.uint8)


class PagedCache:
    """A paged key-value cache: ``k``, ``v`` [num_pages, page_size, Hkv, D]
    (bf16 or fp16; any strides with contiguous D, so a head-major pool works as
    a transposed view), ``table`` int32 [B, max_pages] with contiguous rows, and
    optionally ``weights`` fp32 [num_pages, Hkv, page_size], the accumulated
    attention weight of every cached token. Slot s of sequence b is row
    s % page_size of page table[b, s // page_size]. The tensors are the
    caller's; the pages they hold are written by ``paged_append`` and
    ``cache_evict``."""

    __slots__ = ("_tensors", "packed")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, weights: Optional[torch.Tensor] = None):
        self.packed = (_native or _marshal()).cache(k, v, table, weights)
        self._tensors = (k, v, table, weights)     # what `packed` points to, for good

    @property
    def k(self) -> torch.Tensor:
        return self._tensors[0]

    @property
    def v(self) -> torch.Tensor:
        return self._tensors[1]

    @property
    def table(self) -> torch.Tensor:
        return self._tensors[2]

    @property
    def weights(self) -> Optional[torch.Tensor]:
        return self._tensors[3]

    @property
    def num_pages(self) -> int:
        return self.k.shape[0]

    @property
    def page_size(self) -> int:
        return self.k.shape[1]

    @property
    def Hkv(self) -> int:
        return self.k.shape[2]

    @property
    def capacity(self) -> int:
        """Slots of a sequence."""
        return self.table.shape[1] * self.k.shape[1]


def attn_packed(q, k, v, o, heads: Sequence[int], cu_seqlens, window: Optional[int] = None,
                scale: Optional[float] = None, lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                stream=None):
    """Causal attention of packed prompts: q/o [T,Hq,D], k/v [T,Hkv,D],
    ``cu_seqlens`` int32 [S+1] on the device; writes o[:, heads] (rows of
    sequences) and ``lse`` fp32 [len(heads), T]. ``window`` None: the whole
    prefix. ``ws``: 256 bytes of the caller's; give them to read the call's
    status afterwards (``workspace_status``)."""
    ws = _empty(256, torch.uint8, q, stream) if ws is None else _bytes(ws)
    _call("attn_packed", q, q, k, v, o, _head_bytes(tuple(heads)), cu_seqlens, window, scale, lse, ws,
          None if stream is None else stream.cuda_stream)
    return o


def attn_key_weights(q, k, lse, weights, heads: Sequence[int], cu_seqlens, n_obs: Optional[int] = None,
                     window: Optional[int] = None, scale: Optional[float] = None, ws: Optional[torch.Tensor] = None,
                     stream=None):
    """The attention weight each key of packed prompts got from the last
    ``n_obs`` rows of its sequence (None: every row), summed over the listed
    heads of its KV head, into ``weights`` fp32 [Hkv, T]; ``lse`` fp32
    [len(heads), T] from ``attn_packed``; ``ws`` as there."""
    ws = _empty(256, torch.uint8, q, stream) if ws is None else _bytes(ws)
    _call("attn_key_weights", q, q, k, lse, weights, _head_bytes(tuple(heads)), cu_seqlens, n_obs, window, scale, ws,
          None if stream is None else stream.cuda_stream)
    return weights


def paged_append(cache: PagedCache, k, v, cu_seqlens, pos, weights: Optional[torch.Tensor] = None, stream=None):
    """Puts new tokens into the cache: row t of sequence i (k/v [T,Hkv,D],
    ``cu_seqlens`` int32 [S+1]) goes to slot pos[i] + t - cu_seqlens[i] of
    table row i. ``weights`` fp32 [Hkv,T] starts their accumulated weights
    (None: 0)."""
    _call("paged_append", k, cache.packed, k, v, cu_seqlens, pos, weights,
          None if stream is None else stream.cuda_stream)


def paged_attn_decode(q, cache: PagedCache, lens, o, heads: Sequence[int], window: Optional[int] = None,
                      sink: int = 0, scale: Optional[float] = None, max_len: Optional[int] = None,
                      lse: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None):
    """One new token per sequence over the paged cache: q/o [B,Hq,D], ``lens``
    int32 [B]; attends the slots [0, sink) and the last ``window`` (None: all).
    ``max_len`` (default: the table's capacity) bounds the lengths. ``lse``
    fp32 [B,len(heads)]; ``weights_out`` (like cache.weights, may be it)
    receives cache.weights plus this token's attention weights."""
    if max_len is None:
        max_len = cache.capacity
    if ws is None:
        ws = _empty(decode_workspace_size(q.shape[0], max_len, len(heads), window, sink, weights_out is not None),
                    torch.uint8, q, stream)
    else:
        ws = _bytes(ws)
    _call("paged_attn_decode", q, q, cache.packed, lens, o, _head_bytes(tuple(heads)), window, sink, scale, max_len,
          lse, weights_out, ws, None if stream is None else stream.cuda_stream)
    return o


def decode_workspace_size(B: int, max_len: int, n_heads: int, window: Optional[int], sink: int,
                          with_weights: bool) -> int:
    """Bytes of workspace that ``paged_attn_decode`` needs."""
    return (_native or _marshal()).decode_workspace_size(B, max_len, n_heads, window, sink, with_weights)


def cache_evict(cache: PagedCache, lens, budget: int, sink: int = 0, recent: int = 0,
                out: Optional[PagedCache] = None, idx: Optional[torch.Tensor] = None,
                new_lens: Optional[torch.Tensor] = None, max_len: Optional[int] = None, stream=None):
    """Shrinks the cache to ``budget`` tokens per sequence and KV head: the
    first ``sink``, the last ``recent`` and the others of largest accumulated
    weight, moved to slots 0, 1, ... of ``out`` (default: in place; no page may
    then be shared). Every slot below a length should hold a token: one whose
    page is missing ranks last and, kept all the same, leaves its new slot as it
    was. Afterwards a slot is no longer a position. Returns (idx int32
    [B,Hkv,budget], the kept slots ascending and -1 padded; new_lens int32 [B])."""
    if out is None:
        out = cache
    if idx is None:
        idx = _empty((lens.shape[0], cache.Hkv, max(budget, 0)), torch.int32, lens, stream)
    if new_lens is None:
        new_lens = _empty((lens.shape[0],), torch.int32, lens, stream)
    _call("cache_evict", lens, cache.packed, out.packed, lens, budget, sink, recent, idx, new_lens,
          cache.capacity if max_len is None else max_len, None if stream is None else stream.cuda_stream)
    return idx, new_lens


class PagedLayer:
    """One attention layer over a paged cache: prompts, single tokens, eviction.

    ``heads`` attend everything; with ``window`` the ``streaming`` heads attend
    the last ``window`` tokens and, when decoding, the first ``sink``.
    ``prefill`` runs packed prompts and puts their keys and values (and, if the
    cache has weights, the weights that their last ``n_obs`` queries gave) into
    the cache; ``decode`` appends one token per sequence and attends;
    ``evict`` shrinks the cache in place; from then on the ``window`` of the
    streaming heads counts slots, of which the last ``recent`` and those decoded
    since are the last positions. ``lens`` is the device's record of
    the sequences' lengths, kept by these calls; buffers are kept across calls,
    so the calls of a layer (and replays of graphs that hold them) come one after
    the other: on one stream, or on streams that wait for each other.

    A token beyond the cache's capacity finds no slot: it is dropped, counted in
    ``lens`` (the calls clamp it) until ``evict`` makes room, and reported by
    ``dropped()``. Rows of such a sequence attend what fits, without the token
    itself: evict, or end the sequence, before ``lens`` reaches the capacity.
    """

    def __init__(self, cache: PagedCache, Hq: int, streaming: Sequence[int] = (), window: Optional[int] = None,
                 sink: int = 0, n_obs: Optional[int] = None, scale: Optional[float] = None):
        self.cache, self.Hq, self.n_obs, self.window, self.sink = cache, Hq, n_obs, window, sink
        self.streaming = list(streaming)
        self.full = [h for h in range(Hq) if h not in set(self.streaming)]
        if self.streaming and window is None:
            import long_context_hybrid_b200 as base
            raise base.RtpError("PagedLayer: streaming heads need a window")
        self.scale = scale
        B, dev = cache.table.shape[0], cache.k.device
        self.lens = torch.zeros(B, dtype=torch.int32, device=dev)
        self._dropped = torch.zeros_like(self.lens)   # tokens without a slot, up to the last eviction
        self.cu_decode = torch.arange(B + 1, dtype=torch.int32, device=dev)
        # a status word of its own for every tensor-core call of a prefill: the
        # kernels clear the one they are given
        self.ws_prefill = torch.zeros(len(self._groups()), 2, 256, dtype=torch.uint8, device=dev)
        weighed = cache.weights is not None
        self.ws = torch.empty(max(decode_workspace_size(B, cache.capacity, len(g), w, sink, weighed)
                                  for g, w in self._groups()), dtype=torch.uint8, device=dev)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(dev).synchronize()     # the calls may come on any stream

    def _groups(self):
        """(heads, window) of the two kinds of heads that are there."""
        return [x for x in ((self.full, None), (self.streaming, self.window)) if x[0]]

    def prefill(self, q, k, v, o, cu_seqlens, stream=None):
        """q/o [T,Hq,D], k/v [T,Hkv,D] of B packed prompts (one per table row)."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.cache.k.device)):
            weights = None
            for (heads, window), ws in zip(self._groups(), self.ws_prefill):
                lse = None
                if self.cache.weights is not None:
                    lse = torch.empty(len(heads), q.shape[0], dtype=torch.float32, device=q.device)
                attn_packed(q, k, v, o, heads, cu_seqlens, window, self.scale, lse, ws[0])
                if lse is not None:
                    w = torch.zeros(k.shape[1], k.shape[0], dtype=torch.float32, device=q.device)
                    attn_key_weights(q, k, lse, w, heads, cu_seqlens, self.n_obs, window, self.scale, ws[1])
                    weights = w if weights is None else weights.add_(w)
            self.lens.zero_()
            self._dropped.zero_()
            paged_append(self.cache, k, v, cu_seqlens, self.lens, weights)
            torch.sub(cu_seqlens[1:], cu_seqlens[:-1], out=self.lens)
        return o

    def decode(self, q, k, v, o, stream=None):
        """q/o [B,Hq,D], k/v [B,Hkv,D]: one new token of every sequence."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.cache.k.device)):
            paged_append(self.cache, k, v, self.cu_decode, self.lens)
            self.lens.add_(1)
            for heads, window in self._groups():
                paged_attn_decode(q, self.cache, self.lens, o, heads, window, self.sink if window else 0, self.scale,
                                  weights_out=self.cache.weights, ws=self.ws)
        return o

    def evict(self, budget: int, recent: int, stream=None):
        """Shrinks every sequence to ``budget`` tokens per KV head, keeping the
        ``sink`` first and ``recent`` last; returns the kept slots."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.cache.k.device)):
            idx, new_lens = cache_evict(self.cache, self.lens, budget, self.sink, recent)
            self._dropped.add_(self._beyond())
            self.lens.copy_(new_lens)
        return idx

    def _beyond(self) -> torch.Tensor:
        return (self.lens - self.cache.capacity).clamp_(min=0)

    def dropped(self, stream=None) -> torch.Tensor:
        """int32 [B] on the device: the tokens of each sequence that found no
        slot since its prefill."""
        with torch.cuda.stream(stream or torch.cuda.current_stream(self.cache.k.device)):
            return self._dropped + self._beyond()

    def device_status(self, stream=None) -> int:
        """Synchronises and returns the worst status word of the last prefill's
        attention and key-weight calls (0 = RTP_OK, 4 = RTP_ERR_TIMEOUT: rows of
        ``o`` and weights in the cache are missing). The other calls never wait
        on the device and report nothing there."""
        import long_context_hybrid_b200 as base
        dev = self.cache.k.device
        with torch.cuda.stream(stream or torch.cuda.current_stream(dev)):
            return max(base.workspace_status(ws) for ws in self.ws_prefill.flatten(0, 1))
