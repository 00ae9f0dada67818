"""Plain 64-bit forms of linear attention with a decay for each head and of
layer norm, from their definitions, and the bounds that the GPU tests hold the
kernels to."""

from __future__ import annotations

import math

import torch

U = 2.0 ** -24  # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of the stored type


def decays(g, n):
    """[H, n, n] e^(g (i - j)) for j <= i (1 on the diagonal whatever g is), else 0; [H, n + 1] e^(g m)."""
    m = torch.arange(n + 1, dtype=torch.float64)
    p = torch.where(m == 0, 1.0, torch.exp(g.double()[:, None] * m))
    i = torch.arange(n)
    e = i[:, None] - i[None, :]
    return torch.where(e >= 0, p[:, e.clamp(min=0)], 0.0), p


def attn(q, k, v, g, scale, n, state):
    """One sequence [H, L, d] of n tokens: out and the last state, and the sums of their terms' magnitudes: out's
    from the sequence's own tokens and from the states ahead of its chunks (both at most the whole), the state's."""
    H, L, d = q.shape
    q, k, v = (x[:, :n].double() for x in (q, k, v))
    S = torch.zeros(H, d, d, dtype=torch.float64) if state is None else state.double()
    D, p = decays(g, n)
    out, size = torch.zeros(H, L, d, dtype=torch.float64), torch.zeros(H, L, d, dtype=torch.float64)
    first = p[:, 1:, None]
    out[:, :n] = scale * ((q @ k.mT * D) @ v + first * (q @ S.mT))
    size[:, :n] = scale * ((q.abs() @ k.abs().mT * D) @ v.abs() + first * (q.abs() @ S.abs().mT))
    w = p[:, :n].flip(1)[..., None]
    last = p[:, n, None, None] * S + (v * w).mT @ k
    last_size = p[:, n, None, None] * S.abs() + (v.abs() * w).mT @ k.abs()
    return out, size, last, last_size


def attn_bwd(u, q, k, v, g, scale, n, state, dstate):
    """Gradients of attn for one sequence, each with the sum of its terms' magnitudes."""
    H, L, d = q.shape
    u, q, k, v = (x[:, :n].double() for x in (u, q, k, v))
    zero = torch.zeros(H, d, d, dtype=torch.float64)
    S, R = zero if state is None else state.double(), zero if dstate is None else dstate.double()
    D, p = decays(g, n)
    first, left = scale * p[:, 1:, None], p[:, :n].flip(1)[..., None]
    res = []
    for f in (lambda x: x, torch.abs):
        u1, q1, k1, v1, S1, R1 = (f(x) for x in (u, q, k, v, S, R))
        dp, pr = scale * (u1 @ v1.mT) * D, scale * (q1 @ k1.mT) * D
        dq, dk, dv = (torch.zeros(H, L, d, dtype=torch.float64) for _ in range(3))
        dq[:, :n] = dp @ k1 + first * (u1 @ S1)
        dk[:, :n] = dp.mT @ q1 + left * (v1 @ R1)
        dv[:, :n] = pr.mT @ u1 + left * (k1 @ R1.mT)
        res.append((dq, dk, dv, p[:, n, None, None] * R1 + (u1 * first).mT @ q1))
    return list(zip(*res))


def batch(f, *args, lens, L):
    """f sequence by sequence, its results stacked."""
    rows = []
    for b in range(len(lens)):
        rows.append(f(*[None if x is None else x[b].cpu() for x in args], n=max(0, min(int(lens[b]), L))))
    return rows


def out_bound(value, size, d, L, dtype, rounded):
    """|error| of an output entry.  fp32 sums, in terms of U of the entry's terms: d of a score or of the product with
    the state, 128 of a chunk's products, 2 for each of the L / 32 carries of the state, 16 for decays and scales;
    the tensor cores cut sums off where fp32 arithmetic rounds (a whole step, 2 U).  `rounded`: scores and states
    enter their products in bf16, half a step of each term.  Then the output's own rounding."""
    return HALF[dtype] * value.abs() + size * (2 * (d + 128 + 2 * (L // 32 + 1) + 16) * U + (2.0 ** -8 if rounded else 0.0)) * 1.01 + 1e-37


def state_bound(size, L, split):
    """|error| of a state's entry: sums as above.  `split`: a decayed value is held as two bf16 numbers, off by half a
    step of a half step."""
    return size * (2 * (128 + 2 * (L // 32 + 1) + 16) * U + (2.0 ** -16 if split else 0.0)) * 1.01 + 1e-37


def norm(x, w, b, eps):
    x = x.double()
    c = x - x.mean(-1, keepdim=True)
    z = c / (c.square().mean(-1, keepdim=True) + eps).sqrt()
    return z * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())


def norm_bound(x, w, b, eps, dtype):
    """|error| of a forward entry.  The mean is a sum of D entries (at most 2 log2 D + 40 additions deep: 32 in a
    thread's registers, the rest by halves) and is off by that many U of mean |x|; x - mean carries it and its own
    rounding; the squares' mean has the same depth, each 3 U off and the mean's error besides (to first order it
    drops out of the sum of squares); root, division, product and sum 6 U."""
    x = x.double()
    D = x.shape[-1]
    depth = 2 * math.log2(D + 1) + 40
    n = (x.var(-1, keepdim=True, unbiased=False) + eps).sqrt()
    m = depth * U * x.abs().mean(-1, keepdim=True)
    z = (x - x.mean(-1, keepdim=True)).abs() / n
    dz = m / n * (1 + z) + z * (depth + 10) * U + (m / n) ** 2 * z
    w = torch.ones(D, dtype=torch.float64) if w is None else w.double().abs()
    y = norm(x, None if w is None else w, None, eps).abs()
    bias = 0.0 if b is None else b.double().abs()
    return w * dz + (y + bias) * 4 * U + HALF[dtype] * (z * w + bias) + 1e-37


def norm_bwd(u, x, w, eps):
    """dx, dw, db."""
    D = x.shape[-1]
    x, u = x.double().reshape(-1, D), u.double().reshape(-1, D)
    c = x - x.mean(-1, keepdim=True)
    r = (c.square().mean(-1, keepdim=True) + eps).rsqrt()
    z, t = c * r, u * (1.0 if w is None else w.double())
    dx = r * (t - t.mean(-1, keepdim=True) - z * (t * z).mean(-1, keepdim=True))
    return dx, (u * z).sum(0), u.sum(0)


def norm_bwd_bound(u, x, w, eps, dtype):
    """|error| of dx, dw, db.  z as in norm_bound (dz); t's and t z's means as deep sums; dx's three terms each with
    their own errors, r's 2 depth U; dw and db: z's error of each term, and the sums over N rows (at most N / 608 + 60
    deep)."""
    D = x.shape[-1]
    x, u = x.double().reshape(-1, D), u.double().reshape(-1, D)
    depth = 2 * math.log2(D + 1) + 40
    n = (x.var(-1, keepdim=True, unbiased=False) + eps).sqrt()
    m = depth * U * x.abs().mean(-1, keepdim=True)
    z = (x - x.mean(-1, keepdim=True)).abs() / n
    dz = m / n * (1 + z) + z * (depth + 10) * U + (m / n) ** 2 * z
    t = u.abs() * (1.0 if w is None else w.double().abs())
    mt, mtz = t.mean(-1, keepdim=True), (t * z).mean(-1, keepdim=True)
    dr = (2 * depth + 12) * U + (m / n) ** 2 + m / n * 1e-3
    dx = (t + mt + z * mtz) / n
    err = dx * dr + (mt * depth * U + dz * mtz + z * ((t * dz).mean(-1, keepdim=True) + mtz * depth * U)) / n + dx * 6 * U
    N = x.shape[0]
    rows = (N / 608 + 60) * U
    return (err + HALF[dtype] * dx + 1e-37, (u.abs() * dz).sum(0) + (u.abs() * z).sum(0) * (rows + 2 * U) + 1e-37,
            u.abs().sum(0) * rows + 1e-37)
