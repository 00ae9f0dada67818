"""Plain 64-bit forms of the norm + rotation, the paged cache's attention and
its eviction, loop by loop from their definitions, and the bounds that the
GPU tests hold the kernels to."""

from __future__ import annotations

import math

import torch

U = 2.0 ** -24  # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of the stored type


def pairs_of(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(z, pos, inv_freq, interleaved, back=False):
    """z [B, H, L, d] float64, pos [B, L] int64."""
    y = z.clone()
    if inv_freq is None or len(inv_freq) == 0:
        return y
    a, b = pairs_of(2 * len(inv_freq), interleaved)
    th = pos.double()[:, None, :, None] * inv_freq
    c, s = th.cos(), th.sin() * (-1 if back else 1)
    y[..., a] = z[..., a] * c - z[..., b] * s
    y[..., b] = z[..., b] * c + z[..., a] * s
    return y


def norm_rotate(x, w, pos, inv_freq, interleaved, norm, eps):
    x = x.double()
    if norm:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * (1.0 if w is None else w.double())
    return rotate(x, pos, inv_freq, interleaved)


def norm_rotate_bwd(dy, x, w, pos, inv_freq, interleaved, norm, eps):
    """dx, dw and the sum of dw's absolute terms."""
    x = x.double()
    u = rotate(dy.double(), pos, inv_freq, interleaved, back=True)
    if not norm:
        return u, None, None
    n = (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    g = u * (1.0 if w is None else w.double())
    dx = (g - x * (g * x).sum(-1, keepdim=True) / (x.shape[-1] * n * n)) / n
    t = u * x / n
    return dx, t.sum((0, 1, 2)), t.abs().sum((0, 1, 2))


def rope_bound(y, z, rot, interleaved, out_dtype):
    """|error| of a forward entry.  fp32 arithmetic: the row's sum of squares
    (12 additions deep, a square each), mean, sqrt, division and two products
    give z to 12 U; cosine and sine are off by at most 6 U (2 ulp of sincospif,
    the phase rounded to fp32: pi U); two products and a sum 3 U: 24 U of the
    pair's |z_a| + |z_b| bounds them, then the output's own rounding."""
    m = z.abs().clone()
    if rot:
        a, b = pairs_of(rot, interleaved)
        s = m[..., a] + m[..., b]
        m[..., a], m[..., b] = s, s.clone()
    return HALF[out_dtype] * y.abs() * (1 + 2 ** -8) + 24 * U * m


def rope_bwd_bound(dy, x, w, pos, inv_freq, interleaved, norm, eps, dx, out_dtype):
    """|error| of a dx entry: u to 12 U of its pair (cosine, sine, products),
    then products, the row sums (12 additions deep) and the difference: 40 U
    of (|g| + |x| sum|g x| / (d n^2)) / n, g's magnitude taken over its pair."""
    x = x.double()
    m = dy.double().abs()
    if inv_freq is not None and len(inv_freq):
        a, b = pairs_of(2 * len(inv_freq), interleaved)
        s = m[..., a] + m[..., b]
        m = m.clone()
        m[..., a], m[..., b] = s, s.clone()
    if norm:
        n = (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        g = m * (1.0 if w is None else w.double().abs())
        m = (g + x.abs() * (g * x.abs()).sum(-1, keepdim=True) / (x.shape[-1] * n * n)) / n
    return HALF[out_dtype] * dx.abs() * (1 + 2 ** -8) + 40 * U * m


# ---------------------------------------------------------------- the cache

def slots(pages, table, b, n, page):
    """Rows 0 .. n - 1 of sequence b: [Hk, n, ...]."""
    idx = torch.arange(n)
    return pages[table[b].long()[idx // page], :, idx % page].transpose(0, 1)


def decode(q, k_pages, v_pages, table, lens, scale=None, skip=()):
    """q [B, Hq, d]; returns out, lse (base 2), the list of p [Hk, G, n], and
    a bound of |error| of out and of the p (before out's own rounding).
    skip: pairs (b, slot) that an attention leaves out."""
    B, Hq, d = q.shape
    Hk, page = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hk
    scale = d ** -0.5 if not scale else scale
    out = torch.zeros(B, Hq, d, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    err = torch.zeros(B, Hq, d, dtype=torch.float64)
    ps, pe = [], []
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            ps.append(torch.zeros(Hk, G, 0, dtype=torch.float64))
            pe.append(ps[-1])
            continue
        k, v = slots(k_pages, table, b, n, page).double(), slots(v_pages, table, b, n, page).double()
        qq = q[b].double().view(Hk, G, d)
        s = scale * qq @ k.transpose(1, 2)
        for bb, j in skip:
            if bb == b:
                s[..., j] = -math.inf
        # a score: d products summed in fp32, each step off by at most 2^-23 of the sum of magnitudes so far
        # (tensor cores truncate), q scaled on the way: (d + 8) 2^-23 of scale sum |q k|; a factor e^x is off
        # by the error of x (maximum and lse are such scores) and 2^-22, x = s - max itself rounded: 2^-24 |x|
        ds = (d + 8) * 2.0 ** -23 * scale * (qq.abs() @ k.abs().transpose(1, 2))
        big = torch.where(s.isfinite(), s.abs(), 0.0).amax(-1, keepdim=True)
        rel = 2 * ds.amax(-1, keepdim=True) + 2.0 ** -22 + 2.0 ** -23 * 2 * big
        p = torch.softmax(s, -1)
        live = s.isfinite().any(-1, keepdim=True)
        p = torch.where(live, p, 0.0)
        out[b] = (p @ v).reshape(Hq, d)
        lse[b] = (torch.logsumexp(s, -1) / math.log(2)).reshape(Hq)
        # the sum over n slots: a lane adds at most n / 4 of them, each step off by 2^-23 (plus the joins: 64), and a
        # 16-bit kernel carries p as two bf16 halves: 2^-16
        half = 2.0 ** -16 if q.dtype == torch.bfloat16 else 0.0
        err[b] = ((2 * rel + (64 + n / 4) * 2.0 ** -23 + half) * (p @ v.abs())).reshape(Hq, d)
        ps.append(p)
        pe.append(2 * rel * p)
    return out, lse, ps, err, pe


def evict(weight, table, lens, page, budget, recent, sinks):
    """keep [B, Hk, budget] (int, -1 behind the last) by a plain sort of the slots."""
    B, Hk = len(lens), weight.shape[1]
    keep = torch.full((B, Hk, budget), -1, dtype=torch.int32)
    for b in range(B):
        n = int(lens[b])
        w = slots(weight, table, b, n, page)
        for h in range(Hk):
            if n <= budget:
                keep[b, h, :n] = torch.arange(n)
                continue
            mid = range(sinks, n - recent)
            key = lambda j: (-math.inf if math.isnan(float(w[h, j])) else float(w[h, j]))
            best = sorted(mid, key=lambda j: (-key(j), j))[:budget - sinks - recent]
            keep[b, h] = torch.tensor(sorted([*range(sinks), *best, *range(n - recent, n)]), dtype=torch.int32)
    return keep


def assign(lens, page, rng, extra=0):
    """A shuffled page table for lengths `lens` (-1 behind each sequence's pages), and the pages left over."""
    need = [-(-int(n) // page) for n in lens]
    total = sum(need) + extra
    order = torch.randperm(total, generator=rng).to(torch.int32)
    table = torch.full((len(need), max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table, order[at:], total
