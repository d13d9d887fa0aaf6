"""The 8-bit paged key / value cache: appending tokens, attention over the cached tokens, eviction by
accumulated attention weight.  A thin binding over include/attn_cache_gb300.h, which defines what
each call computes; every step runs in the library's CUDA kernels on the current stream, and
nothing here synchronises, so that all of it can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _capi
from ._capi import AttnCacheAppendArgs, AttnCacheArgs, AttnCacheEvictArgs, AttnCacheFwdArgs, AttnCacheSeqs, AttnError, lib

_DTYPES = {torch.bfloat16: _capi.ATTN_DTYPE_BF16, torch.float32: _capi.ATTN_DTYPE_F32}
_KINDS = {torch.float8_e4m3fn: _capi.ATTN_CACHE_E4M3, torch.int8: _capi.ATTN_CACHE_INT8}


class AttnCache:
    """Handle of a cache's tensors: k and v [num_pages, Hkv, page_size, D] in float8_e4m3fn or int8,
    k_scale and v_scale [num_pages, Hkv] float32, all dense on one CUDA device; ``status`` (made
    here) is the cache's device status area.  The tensors stay the caller's and are used in place.
    ``AttnCache.empty`` allocates them."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "status", "page_size", "_c", "_ref")

    def __init__(self, k, v, k_scale, v_scale):
        where = "AttnCache"
        if k.dtype not in _KINDS or v.dtype != k.dtype:
            raise TypeError(f"{where}: k and v must share dtype float8_e4m3fn or int8")
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError(f"{where}: k and v must both be [num_pages, Hkv, page_size, D]")
        num_pages, Hkv, page_size, D = k.shape
        for name, t, shape, dtype in (("k", k, k.shape, k.dtype), ("v", v, k.shape, k.dtype),
                                      ("k_scale", k_scale, (num_pages, Hkv), torch.float32),
                                      ("v_scale", v_scale, (num_pages, Hkv), torch.float32)):
            if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
                raise ValueError(f"{where}: {name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                                 f"got {t.dtype} {tuple(t.shape)}")
        if page_size not in (16, 32, 64, 128):
            raise ValueError(f"{where}: page_size must be 16, 32, 64 or 128, got {page_size}")
        if D % 16 or not 16 <= D <= 512 or num_pages < 1 or not 1 <= Hkv <= 65535:
            raise ValueError(f"{where}: the head dimension must be a multiple of 16 up to 512, with at least one page and head")
        if k.device.type != "cuda":
            raise ValueError(f"{where}: the cache must be on a CUDA device")
        for t in (v, k_scale, v_scale):
            if t.device != k.device:
                raise ValueError(f"{where}: every tensor must be on {k.device} (got one on {t.device})")
        if k.data_ptr() % 16 or v.data_ptr() % 16:
            raise ValueError(f"{where}: k and v must start on 16-byte boundaries")
        self.k, self.v, self.k_scale, self.v_scale, self.page_size = k, v, k_scale, v_scale, page_size
        self.status = torch.zeros(256, dtype=torch.uint8, device=k.device)
        self._c = AttnCacheArgs(_KINDS[k.dtype], num_pages, page_size, Hkv, D, k.data_ptr(), v.data_ptr(),
                                k_scale.data_ptr(), v_scale.data_ptr(), self.status.data_ptr())
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, num_pages, page_size, Hkv, D, dtype=torch.float8_e4m3fn, device="cuda"):
        """A new cache (its codes and scales are meaningful only where tokens have been appended)."""
        if dtype not in _KINDS:
            raise TypeError("AttnCache: dtype must be float8_e4m3fn or int8")
        shape = (num_pages, Hkv, page_size, D)
        k = torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype)
        v = torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype)
        return cls(k, v, torch.ones((num_pages, Hkv), device=device), torch.ones((num_pages, Hkv), device=device))

    @property
    def num_pages(self):
        return self._c.num_pages

    @property
    def Hkv(self):
        return self._c.Hkv

    @property
    def D(self):
        return self._c.D

    @property
    def device(self):
        return self.k.device


def _check(status: int, where: str):
    if status != _capi.ATTN_OK:
        raise AttnError(status, where)


class _on:
    """Makes the cache's device current for the call (nothing if it is)."""

    __slots__ = ("guard",)

    def __init__(self, device):
        self.guard = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *e):
        if self.guard is not None:
            self.guard.__exit__(*e)


def _seqs(where, cache, B, table, lengths) -> AttnCacheSeqs:
    if table.dim() != 2 or table.shape[0] != B or table.dtype != torch.int32 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"{where}: table must be int32 [{B}, max_pages] with dense rows, got {table.dtype} {tuple(table.shape)}")
    if lengths.dim() != 1 or lengths.shape[0] != B or lengths.dtype != torch.int32 or not lengths.is_contiguous():
        raise ValueError(f"{where}: lengths must be a contiguous int32 tensor of {B} entries, got {lengths.dtype} {tuple(lengths.shape)}")
    _same_device(where, cache, table, lengths)
    if B > 1 and table.stride(0) < table.shape[1]:
        raise ValueError(f"{where}: the rows of table must not overlap")
    return AttnCacheSeqs(B, table.shape[1], table.data_ptr(), table.stride(0), lengths.data_ptr())


def _same_device(where, cache, *tensors):
    device = cache.k.device
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"{where}: every tensor must be on {device} (got one on {t.device})")


def _weights(where, name, t, B, cache, room):
    if t.dim() != 3 or t.dtype != torch.float32 or t.shape[0] != B or t.shape[1] != cache._c.Hkv or t.shape[2] < room \
            or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{where}: {name} must be float32 [{B}, {cache._c.Hkv}, at least {room}] with dense rows, "
                         f"got {t.dtype} {tuple(t.shape)}")


def _rows(where, name, t, cache, shape=None):
    """[B, S, H, D] rows in bfloat16 or float32 with the head dimension dense."""
    if t.dtype not in _DTYPES:
        raise TypeError(f"{where}: {name} must be bfloat16 or float32")
    if t.dim() != 4 or t.shape[3] != cache._c.D or (shape is not None and t.shape != shape):
        want = "[B, S, H, D]" if shape is None else tuple(shape)
        raise ValueError(f"{where}: {name} must be {want} with the cache's D = {cache._c.D}, got {tuple(t.shape)}")
    if t.stride(3) != 1:
        raise ValueError(f"{where}: the head dimension of {name} must be contiguous")


def attn_cache_append(cache: AttnCache, k, v, table, lengths, *, counts=None, weights=None):
    """Quantise the rows k, v [B, S, Hkv, D] (of sequence b the first counts[b]; all S without counts)
    into positions lengths[b], lengths[b] + 1, ... of the sequences whose pages ``table`` [B, max_pages]
    lists.  Returns the new lengths, int32 [B] (``lengths`` is unchanged).  ``weights`` [B, Hkv, >= max_pages
    * page_size] float32: accumulated weights, set to 0 for the new tokens."""
    where = "attn_cache_append"
    _rows(where, "k", k, cache)
    _rows(where, "v", v, cache, k.shape)
    if v.dtype != k.dtype:
        raise TypeError(f"{where}: k and v must share a dtype")
    B, S, H, _ = k.shape
    if H != cache._c.Hkv:
        raise ValueError(f"{where}: k and v must have the cache's {cache._c.Hkv} heads, got {H}")
    s = _seqs(where, cache, B, table, lengths)
    _same_device(where, cache, k, v, counts, weights)
    a = AttnCacheAppendArgs(_DTYPES[k.dtype], S, k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2),
                            v.stride(0), v.stride(1), v.stride(2))
    if counts is not None:
        if counts.shape != lengths.shape or counts.dtype != torch.int32 or not counts.is_contiguous():
            raise ValueError(f"{where}: counts must be a contiguous int32 tensor of {B} entries")
        a.counts = counts.data_ptr()
    if weights is not None:
        _weights(where, "weights", weights, B, cache, table.shape[1] * cache.page_size)
        a.weights, a.weights_stride_b, a.weights_stride_h = weights.data_ptr(), weights.stride(0), weights.stride(1)
    with _on(cache.k.device):
        out = torch.empty_like(lengths)
        a.lengths_out = out.data_ptr()
        _check(lib().attn_cache_append(cache._ref, ctypes.byref(s), ctypes.byref(a),
                                       torch.cuda.current_stream().cuda_stream), where)
    return out


def _fwd_args(where, q, cache, table, lengths, causal, window, softcap, sink, off_by_one, scale, weights, weights_out):
    _rows(where, "q", q, cache)
    B, Sq, Hq, D = q.shape
    if Hq % cache._c.Hkv:
        raise ValueError(f"{where}: q's {Hq} heads must be a multiple of the cache's {cache._c.Hkv}")
    s = _seqs(where, cache, B, table, lengths)
    _same_device(where, cache, q, sink, weights, weights_out)
    a = AttnCacheFwdArgs(_DTYPES[q.dtype], Sq, Hq, q.data_ptr(), q.stride(0), q.stride(1), q.stride(2), bool(causal),
                         int(window), float(softcap), D ** -0.5 if scale is None else float(scale))
    if sink is not None:
        if sink.numel() != Hq or sink.dtype != torch.float32 or not sink.is_contiguous():
            raise ValueError(f"{where}: sink must hold one float32 logit per query head [{Hq}]")
        a.sink = sink.data_ptr()
    if off_by_one:
        a.softmax_type = _capi.ATTN_SOFTMAX_OFF_BY_ONE
    if weights is not None:
        weights_out = weights if weights_out is None else weights_out
        for name, t in (("weights", weights), ("weights_out", weights_out)):
            _weights(where, name, t, B, cache, table.shape[1] * cache.page_size)
        if weights.stride() != weights_out.stride():
            raise ValueError(f"{where}: weights and weights_out must have the same strides")
        a.weights, a.weights_out = weights.data_ptr(), weights_out.data_ptr()
        a.weights_stride_b, a.weights_stride_h = weights.stride(0), weights.stride(1)
    elif weights_out is not None:
        raise ValueError(f"{where}: weights_out needs weights")
    return s, a


def attn_cache_fwd(q, cache: AttnCache, table, lengths, *, causal=False, window=0, softcap=0.0, sink=None,
                   off_by_one=False, scale=None, weights=None, weights_out=None, out=None, lse=None):
    """Attention of the queries q [B, Sq, Hq, D] over the cached tokens of each sequence: returns
    (O [B, Sq, Hq, D] in q's dtype, LSE [B, Hq, Sq] float32), as attn_fwd does over dense keys.  The
    queries stand at the last Sq of the lengths[b] positions (append their keys first; causal
    matters from two queries on).  ``weights`` [B, Hkv, >= max_pages * page_size] float32: every cached key's
    probabilities, summed over the queries and the heads that share its kv head, are added to it
    (or the sum is written to ``weights_out``)."""
    where = "attn_cache_fwd"
    s, a = _fwd_args(where, q, cache, table, lengths, causal, window, softcap, sink, off_by_one, scale, weights, weights_out)
    B, Sq, Hq, _ = q.shape
    _same_device(where, cache, out, lse)
    for name, t, shape, dtype in (("out", out, q.shape, q.dtype), ("lse", lse, (B, Hq, Sq), torch.float32)):
        if t is not None and (tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous()):
            raise ValueError(f"{where}: {name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                             f"got {t.dtype} {tuple(t.shape)}")
    L = lib()
    sr, ar = ctypes.byref(s), ctypes.byref(a)
    with _on(cache.k.device):
        need = L.attn_cache_fwd_workspace_size(cache._ref, sr, ar)
        if need == 0:
            _check(_capi.ATTN_ERR_INVALID, where)
        device = cache.k.device
        O = torch.empty((B, Sq, Hq, cache._c.D), dtype=q.dtype, device=device) if out is None else out
        LSE = torch.empty((B, Hq, Sq), dtype=torch.float32, device=device) if lse is None else lse
        # Scratch of this call alone: the caching allocator hands it on in stream order, and inside a
        # graph capture it belongs to that graph.
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        _check(L.attn_cache_fwd(cache._ref, sr, ar, O.data_ptr(), LSE.data_ptr(), ws.data_ptr(), need,
                                torch.cuda.current_stream().cuda_stream), where)
    return O, LSE


def attn_cache_path_name(q, cache: AttnCache, table, lengths, **kw) -> str:
    """Kernel path attn_cache_fwd takes for these arguments: "mma" (tensor cores) or "simt"."""
    o = dict(causal=False, window=0, softcap=0.0, sink=None, off_by_one=False, scale=None, weights=None, weights_out=None)
    o.update(kw)
    s, a = _fwd_args("attn_cache_path_name", q, cache, table, lengths, **o)
    return lib().attn_cache_path_name(cache._ref, ctypes.byref(s), ctypes.byref(a)).decode()


def attn_cache_evict(cache: AttnCache, table, lengths, weights, table_out, *, keep, recent=0, first=0,
                     kept: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None):
    """Shrink every sequence to at most ``keep`` tokens per kv head: the ``first`` first, the ``recent`` last
    and, of the others, those of largest accumulated weight (weights [B, Hkv, >= max_pages * page_size];
    ties keep the lower position), gathered in order into the pages that table_out [B, >= ceil(keep /
    page_size)] lists.  No page of table_out may be one that the call still reads.  Returns (kept
    [B, Hkv, keep] int32, -1 past the last; new lengths [B] int32; their weights [B, Hkv, keep], 0 past the
    last): table_out and the latter two are the sequences from here on."""
    where = "attn_cache_evict"
    B = lengths.shape[0]
    s = _seqs(where, cache, B, table, lengths)
    keep, recent, first = int(keep), int(recent), int(first)
    if keep < 1 or recent < 0 or first < 0 or first + recent > keep:
        raise ValueError(f"{where}: keep must be at least 1 and at least first + recent")
    _same_device(where, cache, weights, table_out, kept, weights_out)
    _weights(where, "weights", weights, B, cache, table.shape[1] * cache.page_size)
    pages = -(-keep // cache.page_size)
    if table_out.dim() != 2 or table_out.shape[0] != B or table_out.shape[1] < pages or table_out.dtype != torch.int32 \
            or (table_out.shape[1] > 1 and table_out.stride(1) != 1) or (B > 1 and table_out.stride(0) < table_out.shape[1]):
        raise ValueError(f"{where}: table_out must be int32 [{B}, at least {pages}] with dense rows")
    shape = (B, cache._c.Hkv, keep)
    for name, t, dtype in (("kept", kept, torch.int32), ("weights_out", weights_out, torch.float32)):
        if t is not None and (tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous()):
            raise ValueError(f"{where}: {name} must be a contiguous {dtype} tensor of shape {shape}")
    with _on(cache.k.device):
        device = cache.k.device
        kept = torch.empty(shape, dtype=torch.int32, device=device) if kept is None else kept
        weights_out = torch.empty(shape, dtype=torch.float32, device=device) if weights_out is None else weights_out
        lengths_out = torch.empty_like(lengths)
        a = AttnCacheEvictArgs(keep, first, recent, weights.data_ptr(), weights.stride(0), weights.stride(1),
                               table_out.data_ptr(), table_out.stride(0), kept.data_ptr(), lengths_out.data_ptr(),
                               weights_out.data_ptr())
        _check(lib().attn_cache_evict(cache._ref, ctypes.byref(s), ctypes.byref(a),
                                      torch.cuda.current_stream().cuda_stream), where)
    return kept, lengths_out, weights_out


def attn_cache_check_device_status(cache: AttnCache) -> int:
    """Synchronise the current stream and read / clear the cache's status word: ATTN_OK, or ATTN_ERR_DEVICE
    if a call since the last check met a bad page id or length, or a non-finite appended value."""
    with _on(cache.k.device):
        return lib().attn_check_device_status(cache.status.data_ptr(), torch.cuda.current_stream().cuda_stream)
