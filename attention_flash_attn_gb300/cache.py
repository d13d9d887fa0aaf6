"""The 8-bit paged key / value cache: appending tokens, attention over the cached tokens, eviction by
accumulated attention weight.  A thin binding over include/attn_cache_gb300.h, which defines what
each call computes; csrc/binding.cpp checks the arguments and makes the calls.  Every step runs in
the library's CUDA kernels on the current stream, and nothing here synchronises, so that all of it
can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _capi
from ._capi import AttnCacheArgs, lib

_KINDS = {torch.float8_e4m3fn: _capi.ATTN_CACHE_E4M3, torch.int8: _capi.ATTN_CACHE_INT8}


_binding = None


def _calls():
    """The compiled calls of csrc/binding.cpp (raises if they have not been built)."""
    global _binding
    if _binding is None:
        lib()
        try:
            from . import _binding as module
        except ImportError as e:
            raise ImportError(f"the compiled calls of the cache are missing or do not load ({e}): build them with "
                              "attention_flash_attn_gb300.build.build()") from e
        _binding = module
    return _binding


class AttnCache:
    """Handle of a cache's tensors: k and v [num_pages, Hkv, page_size, D] in float8_e4m3fn or int8,
    k_scale and v_scale [num_pages, Hkv] float32, all dense on one CUDA device; ``status`` (made
    here) is the cache's device status area.  The tensors stay the caller's and are used in place.
    ``AttnCache.empty`` allocates them."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "status", "page_size", "num_pages", "Hkv", "D", "device", "_c", "_addr")

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
        self._addr = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, num_pages, page_size, Hkv, D, dtype=torch.float8_e4m3fn, device="cuda"):
        """A new cache (its codes and scales are meaningful only where tokens have been appended)."""
        if dtype not in _KINDS:
            raise TypeError("AttnCache: dtype must be float8_e4m3fn or int8")
        shape = (num_pages, Hkv, page_size, D)
        k = torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype)
        v = torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype)
        return cls(k, v, torch.ones((num_pages, Hkv), device=device), torch.ones((num_pages, Hkv), device=device))


def attn_cache_append(cache: AttnCache, k, v, table, lengths, *, counts=None, weights=None):
    """Quantise the rows k, v [B, S, Hkv, D] (of sequence b the first counts[b]; all S without counts)
    into positions lengths[b], lengths[b] + 1, ... of the sequences whose pages ``table`` [B, max_pages]
    lists.  Returns the new lengths, int32 [B] (``lengths`` is unchanged).  ``weights`` [B, Hkv, >= max_pages
    * page_size] float32: accumulated weights, set to 0 for the new tokens."""
    return _calls().append(cache._addr, cache.k, k, v, table, lengths, counts, weights)


def attn_cache_fwd(q, cache: AttnCache, table, lengths, *, causal=False, window=0, softcap=0.0, sink=None,
                   off_by_one=False, scale=None, weights=None, weights_out=None, out=None, lse=None):
    """Attention of the queries q [B, Sq, Hq, D] over the cached tokens of each sequence: returns
    (O [B, Sq, Hq, D] in q's dtype, LSE [B, Hq, Sq] float32), as attn_fwd does over dense keys.  The
    queries stand at the last Sq of the lengths[b] positions (append their keys first; causal
    matters from two queries on).  ``weights`` [B, Hkv, >= max_pages * page_size] float32: every cached key's
    probabilities, summed over the queries and the heads that share its kv head, are added to it
    (or the sum is written to ``weights_out``)."""
    return _calls().fwd(cache._addr, cache.k, q, table, lengths, causal, window, softcap, sink, off_by_one, scale, weights,
                        weights_out, out, lse)


def attn_cache_path_name(q, cache: AttnCache, table, lengths, *, causal=False, window=0, softcap=0.0, sink=None,
                         off_by_one=False, scale=None, weights=None, weights_out=None) -> str:
    """Kernel path attn_cache_fwd takes for these arguments: "tc" (tcgen05), "mma" (warp-level tensor-core products) or "simt"."""
    return _calls().path(cache._addr, cache.k, q, table, lengths, causal, window, softcap, sink, off_by_one, scale, weights,
                         weights_out)


def attn_cache_evict(cache: AttnCache, table, lengths, weights, table_out, *, keep, recent=0, first=0,
                     kept: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None):
    """Shrink every sequence to at most ``keep`` tokens per kv head: the ``first`` first, the ``recent`` last
    and, of the others, those of largest accumulated weight (weights [B, Hkv, >= max_pages * page_size];
    ties keep the lower position), gathered in order into the pages that table_out [B, >= ceil(keep /
    page_size)] lists.  No page of table_out may be one that the call still reads.  Returns (kept
    [B, Hkv, keep] int32, -1 past the last; new lengths [B] int32; their weights [B, Hkv, keep], 0 past the
    last).  table_out and the new lengths are the sequences from here on; positions, and with them
    windows, count the tokens that are left.  To go on with accumulated weights, give ``weights_out`` rows
    of table_out's width ([B, Hkv, >= table_out.shape[1] * page_size] float32, not overlapping weights nor between its rows): it is
    written up to ``keep``, returned, and what the next append and attention take."""
    return _calls().evict(cache._addr, cache.k, table, lengths, weights, table_out, keep, recent, first, kept, weights_out)


def attn_cache_check_device_status(cache: AttnCache) -> int:
    """Synchronise the current stream and read / clear the cache's status word: ATTN_OK, or ATTN_ERR_DEVICE
    if a call since the last check met a bad page id or length, or a non-finite appended value."""
    with torch.cuda.device(cache.device):
        return lib().attn_check_device_status(cache.status.data_ptr(), torch.cuda.current_stream().cuda_stream)
