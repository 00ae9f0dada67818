"""Query / key norm and rotation (nats_qk_norm_rope, nats_qk_norm_rope_bwd).

Operands are [B, H, L, d] views with any strides but the last, so q and k may
lie inside one projection's output, `qkv.view(B, L, 3, H, d)[:, :, 0].transpose(1, 2)`.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _args, _native
from ._native import RopeDims, check


def rope_inv_freq(rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """float64 [rot / 2]: base^(-2 i / rot), the radians per position of pair i."""
    return torch.tensor([float(base) ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=device)


def _rotation(inv_freq, positions, B, L, device):
    """rot, and the addresses / stride of the frequencies and positions."""
    if inv_freq is None:
        rot, pf = 0, None
    else:
        if inv_freq.dim() != 1:
            raise ValueError(f"inv_freq must have shape (rot / 2,), got {tuple(inv_freq.shape)}")
        pf = _args.need(inv_freq, "inv_freq", torch.float64, None, device)
        rot = 2 * inv_freq.shape[0]
    pp, pb = None, 0
    if positions is not None:
        shape = (L,) if positions.dim() == 1 else (B, L)
        pp = _args.need(positions, "positions", torch.int64, shape, device, contiguous=False)
        if L > 1 and positions.stride(-1) != 1:
            raise ValueError("positions of a sequence must be contiguous")
        pb = 0 if positions.dim() == 1 else positions.stride(0)
    return rot, pf, pp, pb


def _check_pair(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, H, L, d]")
    if q.shape[0] != k.shape[0] or q.shape[2:] != k.shape[2:]:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} differ in more than their heads")


def qk_norm_rope(q, k, w_q=None, w_k=None, inv_freq=None, positions=None, *, pos0: int = 0, interleaved: bool = False,
                 norm: bool = True, eps: float = 1e-6, out_q: Optional[torch.Tensor] = None,
                 out_k: Optional[torch.Tensor] = None, stream=None):
    """RMSNorm of every query and key row and its rotation, in one pass.

    q [B, Hq, L, d], k [B, Hk, L, d] bf16 or fp32 (d 64 or 128); w_q, w_k fp32
    [d] or None (unit); inv_freq float64 [rot / 2] (rope_inv_freq; None: no
    rotation); positions int64 [B, L] or [L], or None: pos0 + t; interleaved:
    pairs (2i, 2i + 1) in place of (i, i + rot / 2); norm=False rotates alone.
    Returns (q', k') in the layer's contiguous [B, H, L, d], or in out_q, out_k
    (any strides but the last; the inputs themselves for in place)."""
    _check_pair(q, k)
    B, Hq, L, d = q.shape
    Hk = k.shape[1]
    dev, dt = q.device, q.dtype
    code = _args.dtype_code(q, "q")
    pq, sq = _args.heads(q, "q", dt, q.shape, dev)
    pk, sk = _args.heads(k, "k", dt, k.shape, dev)
    pwq, pwk = _args.need(w_q, "w_q", torch.float32, (d,), dev), _args.need(w_k, "w_k", torch.float32, (d,), dev)
    rot, pf, pp, pb = _rotation(inv_freq, positions, B, L, dev)
    made = []
    if out_q is None:
        out_q = torch.empty((B, Hq, L, d), dtype=dt, device=dev)
        made.append(out_q)
    if out_k is None:
        out_k = torch.empty((B, Hk, L, d), dtype=dt, device=dev)
        made.append(out_k)
    poq, soq = _args.heads(out_q, "out_q", dt, q.shape, dev)
    pok, sok = _args.heads(out_k, "out_k", dt, k.shape, dev)
    _args.distinct(out_q, "out_q")
    _args.distinct(out_k, "out_k")
    dm = RopeDims(B, L, Hq, Hk, d, rot, int(interleaved), int(norm), code, eps)
    with _args.launch(dev, stream, made) as st:
        check(_native.lib.nats_qk_norm_rope(dm, pq, sq, pk, sk, pwq, pwk, pf, pp, pb, pos0, poq, soq, pok, sok, st),
              "nats_qk_norm_rope")
    return out_q, out_k


def qk_norm_rope_bwd(dq_out, dk_out, q, k, w_q=None, w_k=None, inv_freq=None, positions=None, *, pos0: int = 0,
                     interleaved: bool = False, norm: bool = True, eps: float = 1e-6,
                     dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None, weight_grads: bool = True,
                     workspace=None, stream=None):
    """Gradient of qk_norm_rope: dq_out, dk_out (like its outputs; fp32, as
    hybrid_bwd gives them, or q's dtype) give a dict of dq, dk (q's dtype, or
    the given tensors' own: bf16 or fp32, any strides but the last) and, with
    weight_grads and norm, dw_q, dw_k (fp32 [d]).  q, k and the other arguments
    are the forward's."""
    _check_pair(q, k)
    B, Hq, L, d = q.shape
    Hk = k.shape[1]
    dev, dt, gt = q.device, q.dtype, dq_out.dtype
    code = _args.dtype_code(q, "q")
    gcode = _args.dtype_code(dq_out, "dq_out")
    pq, sq = _args.heads(q, "q", dt, q.shape, dev)
    pk, sk = _args.heads(k, "k", dt, k.shape, dev)
    pgq, sgq = _args.heads(dq_out, "dq_out", gt, q.shape, dev)
    pgk, sgk = _args.heads(dk_out, "dk_out", gt, k.shape, dev)
    pwq, pwk = _args.need(w_q, "w_q", torch.float32, (d,), dev), _args.need(w_k, "w_k", torch.float32, (d,), dev)
    rot, pf, pp, pb = _rotation(inv_freq, positions, B, L, dev)
    made = []
    if dq is None:
        dq = torch.empty((B, Hq, L, d), dtype=dt if dk is None else dk.dtype, device=dev)
        made.append(dq)
    if dk is None:
        dk = torch.empty((B, Hk, L, d), dtype=dq.dtype, device=dev)
        made.append(dk)
    xcode = _args.dtype_code(dq, "dq")
    pdq, sdq = _args.heads(dq, "dq", dq.dtype, q.shape, dev)
    pdk, sdk = _args.heads(dk, "dk", dq.dtype, k.shape, dev)
    _args.distinct(dq, "dq")
    _args.distinct(dk, "dk")
    dm = RopeDims(B, L, Hq, Hk, d, rot, int(interleaved), int(norm), code, eps)
    res = {"dq": dq, "dk": dk}
    pws, nws, pdw = None, 0, (None, None)
    if weight_grads and norm:
        dw = torch.empty((2, d), dtype=torch.float32, device=dev)
        res["dw_q"], res["dw_k"] = dw[0], dw[1]
        pdw = (dw.data_ptr(), dw.data_ptr() + 4 * d)
        ws, new = _args.workspace(workspace, _native.lib.nats_qk_norm_rope_bwd_workspace_size(dm), dev)
        pws, nws = ws.data_ptr(), ws.numel()
        made.append(dw)
        if new:
            made.append(ws)
    with _args.launch(dev, stream, made) as st:
        check(_native.lib.nats_qk_norm_rope_bwd(dm, gcode, xcode, pgq, sgq, pgk, sgk, pq, sq, pk, sk, pwq, pwk, pf, pp,
                                                pb, pos0, pdq, sdq, pdk, sdk, *pdw, pws, nws, st),
              "nats_qk_norm_rope_bwd")
    return res
