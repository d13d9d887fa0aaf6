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
_I32, _F32 = torch.int32, torch.float32
_current_device = torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)  # the same handle without building a Stream object
_KINDS = {torch.float8_e4m3fn: _capi.ATTN_CACHE_E4M3, torch.int8: _capi.ATTN_CACHE_INT8}


class AttnCache:
    """Handle of a cache's tensors: k and v [num_pages, Hkv, page_size, D] in float8_e4m3fn or int8,
    k_scale and v_scale [num_pages, Hkv] float32, all dense on one CUDA device; ``status`` (made
    here) is the cache's device status area.  The tensors stay the caller's and are used in place.
    ``AttnCache.empty`` allocates them."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "status", "page_size", "num_pages", "Hkv", "D", "device", "_c", "_ref")

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
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.Hkv, self.page_size, self.D, self.device = num_pages, Hkv, page_size, D, k.device
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


def _launch(where, cache, fn, *args):
    """fn(*args, stream) on the current stream of the cache's device, which the library wants current."""
    index = cache.device.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != _capi.ATTN_OK:
        raise AttnError(status, where)


def _seqs(where, cache, B, table, lengths) -> AttnCacheSeqs:
    shape, device = table.shape, cache.device
    if len(shape) != 2 or shape[0] != B or table.dtype != _I32:
        raise ValueError(f"{where}: table must be int32 [{B}, max_pages], got {table.dtype} {tuple(shape)}")
    row, col = table.stride()
    if (col != 1 and shape[1] > 1) or (row < shape[1] and B > 1):
        raise ValueError(f"{where}: the rows of table must be dense and not overlap")
    if lengths.dtype != _I32 or tuple(lengths.shape) != (B,) or not lengths.is_contiguous():
        raise ValueError(f"{where}: lengths must be a contiguous int32 tensor of {B} entries, got {lengths.dtype} {tuple(lengths.shape)}")
    if table.device != device or lengths.device != device:
        _same_device(where, cache, table, lengths)
    return AttnCacheSeqs(B, shape[1], table.data_ptr(), row, lengths.data_ptr())


def _same_device(where, cache, *tensors):
    device = cache.device
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"{where}: every tensor must be on {device} (got one on {t.device})")


def _weights(where, name, t, B, cache, room):
    """Strides of accumulated weights, checked."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or t.dtype != _F32 or shape[0] != B or shape[1] != cache.Hkv or shape[2] < room \
            or (stride[2] != 1 and shape[2] > 1):
        raise ValueError(f"{where}: {name} must be float32 [{B}, {cache.Hkv}, at least {room}] with dense rows, "
                         f"got {t.dtype} {tuple(shape)}")
    _same_device(where, cache, t)
    return stride


def _rows(where, name, t, cache):
    """dtype code, shape and strides of [B, S, H, D] rows in bfloat16 or float32 with the head dimension dense."""
    dtype = _DTYPES.get(t.dtype)
    if dtype is None:
        raise TypeError(f"{where}: {name} must be bfloat16 or float32")
    shape = t.shape
    if len(shape) != 4 or shape[3] != cache.D:
        raise ValueError(f"{where}: {name} must be [B, S, H, D] with the cache's D = {cache.D}, got {tuple(shape)}")
    stride = t.stride()
    if stride[3] != 1:
        raise ValueError(f"{where}: the head dimension of {name} must be contiguous")
    if t.device != cache.device:
        _same_device(where, cache, t)
    return dtype, shape, stride


def attn_cache_append(cache: AttnCache, k, v, table, lengths, *, counts=None, weights=None):
    """Quantise the rows k, v [B, S, Hkv, D] (of sequence b the first counts[b]; all S without counts)
    into positions lengths[b], lengths[b] + 1, ... of the sequences whose pages ``table`` [B, max_pages]
    lists.  Returns the new lengths, int32 [B] (``lengths`` is unchanged).  ``weights`` [B, Hkv, >= max_pages
    * page_size] float32: accumulated weights, set to 0 for the new tokens."""
    where = "attn_cache_append"
    dtype, (B, S, H, _), ks = _rows(where, "k", k, cache)
    vdtype, vshape, vs = _rows(where, "v", v, cache)
    if vdtype != dtype:
        raise TypeError(f"{where}: k and v must share a dtype")
    if vshape != k.shape:
        raise ValueError(f"{where}: v must be {tuple(k.shape)}, got {tuple(vshape)}")
    if H != cache.Hkv:
        raise ValueError(f"{where}: k and v must have the cache's {cache.Hkv} heads, got {H}")
    s = _seqs(where, cache, B, table, lengths)
    cp = wp = None
    wb = wh = 0
    if counts is not None:
        if counts.shape != lengths.shape or counts.dtype != _I32 or not counts.is_contiguous():
            raise ValueError(f"{where}: counts must be a contiguous int32 tensor of {B} entries")
        _same_device(where, cache, counts)
        cp = counts.data_ptr()
    if weights is not None:
        wb, wh, _ = _weights(where, "weights", weights, B, cache, table.shape[1] * cache.page_size)
        wp = weights.data_ptr()
    out = torch.empty_like(lengths)
    a = AttnCacheAppendArgs(dtype, S, k.data_ptr(), v.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], cp, out.data_ptr(),
                            wp, wb, wh)
    _launch(where, cache, lib().attn_cache_append, cache._ref, s, a)
    return out


def _fwd_args(where, q, cache, table, lengths, causal, window, softcap, sink, off_by_one, scale, weights, weights_out):
    dtype, (B, Sq, Hq, D), qs = _rows(where, "q", q, cache)
    if Hq % cache.Hkv:
        raise ValueError(f"{where}: q's {Hq} heads must be a multiple of the cache's {cache.Hkv}")
    s = _seqs(where, cache, B, table, lengths)
    sp = wp = op = None
    wb = wh = 0
    if sink is not None:
        if sink.numel() != Hq or sink.dtype != _F32 or not sink.is_contiguous():
            raise ValueError(f"{where}: sink must hold one float32 logit per query head [{Hq}]")
        _same_device(where, cache, sink)
        sp = sink.data_ptr()
    if weights is not None:
        room = table.shape[1] * cache.page_size
        stride = _weights(where, "weights", weights, B, cache, room)
        if weights_out is None:
            weights_out = weights
        elif _weights(where, "weights_out", weights_out, B, cache, room) != stride:
            raise ValueError(f"{where}: weights and weights_out must have the same strides")
        wp, op, wb, wh = weights.data_ptr(), weights_out.data_ptr(), stride[0], stride[1]
    elif weights_out is not None:
        raise ValueError(f"{where}: weights_out needs weights")
    return s, AttnCacheFwdArgs(dtype, Sq, Hq, q.data_ptr(), qs[0], qs[1], qs[2], 1 if causal else 0, window, softcap,
                               D ** -0.5 if scale is None else scale, sp,
                               _capi.ATTN_SOFTMAX_OFF_BY_ONE if off_by_one else _capi.ATTN_SOFTMAX_DEFAULT, wp, op, wb, wh)


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
    B, Sq, Hq, _ = shape = q.shape
    device = cache.device
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=device)
    elif out.shape != shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError(f"{where}: out must be a contiguous {q.dtype} tensor of shape {tuple(shape)}, got {out.dtype} {tuple(out.shape)}")
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=_F32, device=device)
    elif tuple(lse.shape) != (B, Hq, Sq) or lse.dtype != _F32 or not lse.is_contiguous():
        raise ValueError(f"{where}: lse must be a contiguous float32 tensor of shape {(B, Hq, Sq)}, got {lse.dtype} {tuple(lse.shape)}")
    _same_device(where, cache, out, lse)
    L = lib()
    need = L.attn_cache_fwd_workspace_size(cache._ref, s, a)
    if need == 0:
        raise AttnError(_capi.ATTN_ERR_INVALID, where)
    # Scratch of this call alone: the caching allocator hands it on in stream order, and inside a graph
    # capture it belongs to that graph.
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    _launch(where, cache, L.attn_cache_fwd, cache._ref, s, a, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), need)
    return out, lse


def attn_cache_path_name(q, cache: AttnCache, table, lengths, **kw) -> str:
    """Kernel path attn_cache_fwd takes for these arguments: "mma" (tensor cores) or "simt"."""
    o = dict(causal=False, window=0, softcap=0.0, sink=None, off_by_one=False, scale=None, weights=None, weights_out=None)
    o.update(kw)
    s, a = _fwd_args("attn_cache_path_name", q, cache, table, lengths, **o)
    return lib().attn_cache_path_name(cache._ref, s, a).decode()


def attn_cache_evict(cache: AttnCache, table, lengths, weights, table_out, *, keep, recent=0, first=0,
                     kept: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None):
    """Shrink every sequence to at most ``keep`` tokens per kv head: the ``first`` first, the ``recent`` last
    and, of the others, those of largest accumulated weight (weights [B, Hkv, >= max_pages * page_size];
    ties keep the lower position), gathered in order into the pages that table_out [B, >= ceil(keep /
    page_size)] lists.  No page of table_out may be one that the call still reads.  Returns (kept
    [B, Hkv, keep] int32, -1 past the last; new lengths [B] int32; their weights [B, Hkv, keep], 0 past the
    last): table_out and the latter two are the sequences from here on."""
    where = "attn_cache_evict"
    B = lengths.numel()
    s = _seqs(where, cache, B, table, lengths)
    keep, recent, first = int(keep), int(recent), int(first)
    if keep < 1 or recent < 0 or first < 0 or first + recent > keep:
        raise ValueError(f"{where}: keep must be at least 1 and at least first + recent")
    wb, wh, _ = _weights(where, "weights", weights, B, cache, table.shape[1] * cache.page_size)
    pages = -(-keep // cache.page_size)
    width, row = table_out.shape, table_out.stride()
    if len(width) != 2 or width[0] != B or width[1] < pages or table_out.dtype != _I32 or (row[1] != 1 and width[1] > 1) \
            or (row[0] < width[1] and B > 1):
        raise ValueError(f"{where}: table_out must be int32 [{B}, at least {pages}] with dense rows")
    _same_device(where, cache, table_out, kept, weights_out)
    shape, device = (B, cache.Hkv, keep), cache.device
    for name, t, dtype in (("kept", kept, _I32), ("weights_out", weights_out, _F32)):
        if t is not None and (tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous()):
            raise ValueError(f"{where}: {name} must be a contiguous {dtype} tensor of shape {shape}")
    if kept is None:
        kept = torch.empty(shape, dtype=_I32, device=device)
    if weights_out is None:
        weights_out = torch.empty(shape, dtype=_F32, device=device)
    lengths_out = torch.empty_like(lengths)
    a = AttnCacheEvictArgs(keep, first, recent, weights.data_ptr(), wb, wh, table_out.data_ptr(), row[0], kept.data_ptr(),
                           lengths_out.data_ptr(), weights_out.data_ptr())
    _launch(where, cache, lib().attn_cache_evict, cache._ref, s, a)
    return kept, lengths_out, weights_out


def attn_cache_check_device_status(cache: AttnCache) -> int:
    """Synchronise the current stream and read / clear the cache's status word: ATTN_OK, or ATTN_ERR_DEVICE
    if a call since the last check met a bad page id or length, or a non-finite appended value."""
    index = cache.device.index
    with torch.cuda.device(index):
        return lib().attn_check_device_status(cache.status.data_ptr(), _raw_stream(index))
