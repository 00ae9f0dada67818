"""The paged key / value cache: append, attention of one new token, eviction
(nats_paged_append, nats_paged_decode, nats_paged_evict).  The checks of the
operators' arguments are in csrc/binding.cpp."""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _native

_CODES = {torch.bfloat16: _native.NATS_BF16, torch.float32: _native.NATS_F32}


def _field(t, name, dtype, shape, device):
    """The address of one of the cache's tensors."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _kept(i, name):
    """One of the cache's tensors: it may be changed in place (also by +=), not put in another's place."""
    def get(self):
        return self._t[i]

    def put(self, t):
        if t is not self._t[i]:
            raise AttributeError(f"a cache keeps the {name} that it was made with; change it in place ({name}.copy_)")

    return property(get, put)


class PagedCache:
    """A pool of pages shared by B sequences (nats_paged_cache): k_pages,
    v_pages [n_pages, Hk, page, d] bf16 or fp32; table int32 [B, max_pages],
    the page of every `page` slots of a sequence; lens int32 [B], the slots in
    use; weight fp32 [n_pages, Hk, page] or None, the attention weight that
    paged_decode(accumulate=True) sums and paged_evict goes by; err int32 [1],
    set when a call met a bad table entry or length (`check()` reads it).

    The caller assigns the pages and changes table and lens in place; the
    cache's tensors themselves stay the ones it was made with."""

    def __init__(self, k_pages, v_pages, table, lens, *, weight=None):
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [n_pages, Hk, page, d]")
        n, Hk, page, d = k_pages.shape
        if table.dim() != 2:
            raise ValueError("table must be [B, max_pages]")
        B, most = table.shape
        if not k_pages.is_cuda:
            raise ValueError("k_pages must be a CUDA tensor")
        if k_pages.dtype not in _CODES:
            raise TypeError(f"k_pages must be bfloat16 or float32, got {k_pages.dtype}")
        dev = k_pages.device
        err = torch.zeros((1,), dtype=torch.int32, device=dev)
        self._t = (k_pages, v_pages, table, lens, weight, err)
        self.device, self.dtype = dev, k_pages.dtype
        self.n_pages, self.Hk, self.page, self.d, self.B, self.max_pages = n, Hk, page, d, B, most
        self._c = _native.PagedCache(
            _field(k_pages, "k_pages", k_pages.dtype, None, dev), _field(v_pages, "v_pages", k_pages.dtype, k_pages.shape, dev),
            _field(weight, "weight", torch.float32, (n, Hk, page), dev), _field(table, "table", torch.int32, None, dev),
            _field(lens, "lens", torch.int32, (B,), dev), err.data_ptr(), n, page, Hk, d, B, most, _CODES[k_pages.dtype])
        self._addr, self._dev = ctypes.addressof(self._c), dev.index

    k_pages, v_pages, table, lens, weight, err = (
        _kept(i, name) for i, name in enumerate(("k_pages", "v_pages", "table", "lens", "weight", "err")))

    @classmethod
    def empty(cls, n_pages: int, page: int, Hk: int, d: int, B: int, max_pages: int, *, dtype=torch.bfloat16,
              weight: bool = False, device="cuda") -> "PagedCache":
        """A new pool with no page assigned (table -1) and lengths 0."""
        z = dict(device=device)
        return cls(torch.zeros((n_pages, Hk, page, d), dtype=dtype, **z),
                   torch.zeros((n_pages, Hk, page, d), dtype=dtype, **z),
                   torch.full((B, max_pages), -1, dtype=torch.int32, **z), torch.zeros((B,), dtype=torch.int32, **z),
                   weight=torch.zeros((n_pages, Hk, page), dtype=torch.float32, **z) if weight else None)

    def _used_on(self, stream) -> None:
        """The cache may be freed before a call on `stream` has run: its memory is not handed out again until then."""
        if stream is not None:
            for t in self._t:
                if t is not None:
                    t.record_stream(stream)

    def check(self) -> None:
        """Raises if a call since the cache was made met a table entry outside
        the pool, a length outside the table or an append behind it
        (synchronises with the device)."""
        if int(self.err.item()) != 0:
            raise _native.NatsError(8, "paged cache (a table entry or length out of range)")


def paged_workspace_size(cache: PagedCache, *, Hq: int = 0, accumulate: bool = False, budget: int = 0) -> int:
    """Bytes of workspace that serve paged_decode with Hq query heads and
    paged_evict to `budget` (0 when a size is not supported)."""
    for name, v in (("Hq", Hq), ("budget", budget)):
        if not -(1 << 31) <= v < 1 << 31:
            raise ValueError(f"{name} is out of range")
    a = int(_native.lib.nats_paged_decode_workspace_size(cache._c, Hq, int(accumulate)))
    b = int(_native.lib.nats_paged_evict_workspace_size(cache._c, budget))
    return max(a, b) if a and b else 0


def paged_append(cache: PagedCache, k, v, *, start=None, n_new=None, q=None, out_q: Optional[torch.Tensor] = None,
                 norm: bool = False, w_q=None, w_k=None, inv_freq=None, positions=None, interleaved: bool = False,
                 eps: float = 1e-6, stream=None):
    """New tokens' keys and values k, v [B, Hk, T, d] (any strides but the
    last) into the cache: token t < n_new[b] (int32 [B]; None: all T) goes to
    slot start[b] + t (int32 [B]; None: cache.lens).  With norm / inv_freq the
    keys, and q [B, Hq, T, d] when given, take qk_norm_rope's norm and rotation
    on the way (at `positions`, int64 [B, T], or their slots).  Returns q' (in
    out_q, whose rows from n_new[b] on are left as they were, or in a new
    tensor, zero there), or None without q.  cache.lens is not changed."""
    cache._used_on(stream)
    return _native.operators.paged_append(cache._addr, cache._dev, k, v, start, n_new, q, out_q, norm, w_q, w_k, inv_freq,
                                          positions, interleaved, eps, stream)


def paged_decode(cache: PagedCache, q, *, scale: float = 0.0, accumulate: bool = False, return_lse: bool = False,
                 out=None, workspace=None, stream=None):
    """Attention of one new token of each sequence, q [B, Hq, d], over its
    slots j < cache.lens[b]; query head h reads key head h / (Hq / Hk).
    Returns out [B, Hq, d], or (out, lse) with lse fp32 [B, Hq] in base 2.
    accumulate adds each slot's attention weight, summed over the query heads
    of its key head, to cache.weight (no page may then be in the table twice).  workspace: uint8 tensor of
    paged_workspace_size(cache, Hq=Hq, accumulate=accumulate) bytes, or None."""
    if accumulate and cache.weight is None:
        raise ValueError("accumulate needs a cache with weights")
    cache._used_on(stream)
    return _native.operators.paged_decode(cache._addr, cache._dev, q, scale, accumulate, return_lse, out, workspace, stream)


def paged_evict(cache: PagedCache, out_table, budget: int, *, recent: int = 0, sinks: int = 0, lens_out=None,
                return_keep: bool = False, workspace=None, stream=None):
    """Of every sequence with more than `budget` slots, every key head keeps
    the first `sinks`, the last `recent` and the heaviest (cache.weight) of
    those between, `budget` in all; shorter ones keep all.  The kept rows are
    copied in order to the pages of out_table (int32 [B, m], pages of the same
    pool that no sequence uses).  Returns the new lengths (int32 [B]), or
    (keep, lengths) with keep int32 [B, Hk, budget], the kept slots, -1 behind
    the last.  The caller then puts out_table and the lengths into the cache
    and frees the old pages."""
    if cache.weight is None:
        raise ValueError("eviction needs a cache with weights")
    cache._used_on(stream)
    return _native.operators.paged_evict(cache._addr, cache._dev, out_table, budget, recent, sinks, lens_out, return_keep,
                                         workspace, stream)
