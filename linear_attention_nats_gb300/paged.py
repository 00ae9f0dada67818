"""The paged key / value cache: append, attention of one new token, eviction
(nats_paged_append, nats_paged_decode, nats_paged_evict)."""

from __future__ import annotations

from typing import Optional

import torch

from . import _args, _native
from .rope import _rotation


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
        dev = _args.cuda_index(k_pages, "k_pages")
        code = _args.dtype_code(k_pages, "k_pages")
        pk = _args.need(k_pages, "k_pages", k_pages.dtype, None, dev)
        pv = _args.need(v_pages, "v_pages", k_pages.dtype, k_pages.shape, dev)
        pt = _args.need(table, "table", torch.int32, None, dev)
        pl = _args.need(lens, "lens", torch.int32, (B,), dev)
        pw = _args.need(weight, "weight", torch.float32, (n, Hk, page), dev)
        self._t = (k_pages, v_pages, table, lens, weight, torch.zeros((1,), dtype=torch.int32, device=dev))
        self._dev, self.device, self.dtype = dev, k_pages.device, k_pages.dtype
        self.n_pages, self.Hk, self.page, self.d, self.B, self.max_pages = n, Hk, page, d, B, most
        self._c = _native.PagedCache(pk, pv, pw, pt, pl, self._t[5].data_ptr(), n, page, Hk, d, B, most, code)

    k_pages = property(lambda self: self._t[0])
    v_pages = property(lambda self: self._t[1])
    table = property(lambda self: self._t[2])
    lens = property(lambda self: self._t[3])
    weight = property(lambda self: self._t[4])
    err = property(lambda self: self._t[5])

    @classmethod
    def empty(cls, n_pages: int, page: int, Hk: int, d: int, B: int, max_pages: int, *, dtype=torch.bfloat16,
              weight: bool = False, device="cuda") -> "PagedCache":
        """A new pool with no page assigned (table -1) and lengths 0."""
        z = dict(device=device)
        return cls(torch.zeros((n_pages, Hk, page, d), dtype=dtype, **z),
                   torch.zeros((n_pages, Hk, page, d), dtype=dtype, **z),
                   torch.full((B, max_pages), -1, dtype=torch.int32, **z), torch.zeros((B,), dtype=torch.int32, **z),
                   weight=torch.zeros((n_pages, Hk, page), dtype=torch.float32, **z) if weight else None)

    def check(self) -> None:
        """Raises if a call since the cache was made met a table entry outside
        the pool, a length outside the table or an append behind it
        (synchronises with the device)."""
        if int(self.err.item()) != 0:
            raise _native.NatsError(8, "paged cache (a table entry or length out of range)")


def paged_workspace_size(cache: PagedCache, *, Hq: int = 0, accumulate: bool = False, budget: int = 0) -> int:
    """Bytes of workspace that serve paged_decode with Hq query heads and
    paged_evict to `budget` (0 when a size is not supported)."""
    _args.int32(Hq=Hq, budget=budget)
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
    if k.dim() != 4:
        raise ValueError("k must be [B, Hk, T, d]")
    B, Hk, T, d = k.shape
    dev, dt = cache._dev, cache.dtype
    if (B, Hk, d) != (cache.B, cache.Hk, cache.d):
        raise ValueError(f"k must be [{cache.B}, {cache.Hk}, T, {cache.d}], got {tuple(k.shape)}")
    ks = k.shape
    pk, sk = _args.heads(k, "k", dt, ks, dev)
    pv, sv = _args.heads(v, "v", dt, ks, dev)
    ps = _args.need(start, "start", torch.int32, (B,), dev)
    pn = _args.need(n_new, "n_new", torch.int32, (B,), dev)
    pwq, pwk = _args.need(w_q, "w_q", torch.float32, (d,), dev), _args.need(w_k, "w_k", torch.float32, (d,), dev)
    rot, pf, pp, pb = _rotation(inv_freq, positions, B, T, dev)
    Hq, made = 0, []
    pq = sq = poq = soq = None
    if q is not None:
        qs = q.shape
        if len(qs) != 4 or qs[0] != B or qs[2] != T or qs[3] != d:
            raise ValueError(f"q must be [{B}, Hq, {T}, {d}], got {tuple(qs)}")
        Hq = qs[1]
        pq, sq = _args.heads(q, "q", dt, qs, dev)
        if out_q is None:
            out_q = (torch.empty if n_new is None else torch.zeros)(qs, dtype=dt, device=dev)
            made.append(out_q)
        poq, soq = _args.heads_out(out_q, "out_q", dt, qs, dev)
    dm = _args.rope_dims(B, T, Hq, Hk, d, rot, interleaved, norm, cache._c.dtype, eps)
    _args.call(_native.lib.nats_paged_append, "nats_paged_append", dev, stream, made, cache._c, dm, pq, sq, pk, sk, pv,
               sv, pwq, pwk, pf, ps, pn, pp, pb, poq, soq)
    return out_q


def paged_decode(cache: PagedCache, q, *, scale: float = 0.0, accumulate: bool = False, return_lse: bool = False,
                 out=None, workspace=None, stream=None):
    """Attention of one new token of each sequence, q [B, Hq, d], over its
    slots j < cache.lens[b]; query head h reads key head h / (Hq / Hk).
    Returns out [B, Hq, d], or (out, lse) with lse fp32 [B, Hq] in base 2.
    accumulate adds each slot's attention weight, summed over the query heads
    of its key head, to cache.weight.  workspace: uint8 tensor of
    paged_workspace_size(cache, Hq=Hq, accumulate=accumulate) bytes, or None."""
    dev, dt, c = cache._dev, cache.dtype, cache._c
    qs = q.shape
    if len(qs) != 3 or qs[0] != cache.B or qs[2] != cache.d:
        raise ValueError(f"q must be [{cache.B}, Hq, {cache.d}], got {tuple(qs)}")
    if q.dtype is not dt or q.get_device() != dev:
        _args.refuse(q, "q", dt, None, dev)
    qb, qh, qe = q.stride()
    if qe != 1 and q.numel() > 0:
        raise ValueError("q: the entries of a row must be contiguous")
    if accumulate and cache.weight is None:
        raise ValueError("accumulate needs a cache with weights")
    made, Hq, lib = [], qs[1], _native.lib
    if out is None:
        out = torch.empty(qs, dtype=dt, device=dev)
        made.append(out)
    po, lse, pl = _args.need(out, "out", dt, qs, dev), None, None
    if return_lse:
        lse = torch.empty(qs[:2], dtype=torch.float32, device=dev)
        pl = lse.data_ptr()
        made.append(lse)
    if workspace is None:
        workspace = torch.empty(lib.nats_paged_decode_workspace_size(c, Hq, accumulate), dtype=torch.uint8, device=dev)
        made.append(workspace)
    pw = _args.need(workspace, "workspace", torch.uint8, None, dev)
    _args.call(lib.nats_paged_decode, "nats_paged_decode", dev, stream, made, c, Hq, scale, q.data_ptr(), qb, qh, po, pl,
               accumulate, pw, workspace.numel())
    return (out, lse) if return_lse else out


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
    dev, c, lib = cache._dev, cache._c, _native.lib
    if cache.weight is None:
        raise ValueError("eviction needs a cache with weights")
    if out_table.dim() != 2 or out_table.shape[0] != cache.B:
        raise ValueError(f"out_table must be [{cache.B}, pages], got {tuple(out_table.shape)}")
    _args.int32(budget=budget, recent=recent, sinks=sinks)
    pt = _args.need(out_table, "out_table", torch.int32, None, dev)
    made = []
    if lens_out is None:
        lens_out = torch.empty((cache.B,), dtype=torch.int32, device=dev)
        made.append(lens_out)
    pl = _args.need(lens_out, "lens_out", torch.int32, (cache.B,), dev)
    keep, pk = None, None
    if return_keep:
        keep = torch.empty((cache.B, cache.Hk, max(budget, 0)), dtype=torch.int32, device=dev)
        pk = keep.data_ptr()
        made.append(keep)
    if workspace is None:
        workspace = torch.empty(lib.nats_paged_evict_workspace_size(c, budget), dtype=torch.uint8, device=dev)
        made.append(workspace)
    pw = _args.need(workspace, "workspace", torch.uint8, None, dev)
    _args.call(lib.nats_paged_evict, "nats_paged_evict", dev, stream, made, c, pt, out_table.shape[1], budget, recent,
               sinks, pl, pk, pw, workspace.numel())
    return (keep, lens_out) if return_keep else lens_out
