"""Query / key norm and rotation (nats_qk_norm_rope, nats_qk_norm_rope_bwd).

Operands are [B, H, L, d] views with any strides but the last, so q and k may
lie inside one projection's output, `qkv.view(B, L, 3, H, d)[:, :, 0].transpose(1, 2)`.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _args, _native


def rope_inv_freq(rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """float64 [rot / 2]: base^(-2 i / rot), the radians per position of pair i."""
    return torch.tensor([float(base) ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=device)


def _rotation(inv_freq, positions, B, L, device):
    """rot, and the addresses / stride of the frequencies and positions."""
    rot, pf, pp, pb = 0, None, None, 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError(f"inv_freq must have shape (rot / 2,), got {tuple(inv_freq.shape)}")
        pf = _args.need(inv_freq, "inv_freq", torch.float64, None, device)
        rot = 2 * inv_freq.shape[0]
    if positions is not None:
        shape = (B, L) if positions.dim() == 2 else (L,)
        if positions.dtype is not torch.int64 or positions.get_device() != device or positions.shape != shape:
            _args.refuse(positions, "positions", torch.int64, shape, device)
        st = positions.stride()
        if st[-1] != 1 and L > 1:
            raise ValueError("positions of a sequence must be contiguous")
        pp, pb = positions.data_ptr(), st[0] if len(st) == 2 else 0
    return rot, pf, pp, pb


def _pos0(pos0):
    if not -(1 << 62) <= pos0 < 1 << 62:
        raise ValueError(f"pos0 = {pos0} is out of range")
    return pos0


def _pair(q, k):
    """The shapes of q and k, which differ in their heads alone."""
    qs, ks = q.shape, k.shape
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("q and k must be [B, H, L, d]")
    if ks != (qs[0], ks[1], qs[2], qs[3]):
        raise ValueError(f"q {tuple(qs)} and k {tuple(ks)} differ in more than their heads")
    return qs, ks


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
    qs, ks = _pair(q, k)
    B, Hq, L, d = qs
    dev, dt = _args.cuda_index(q, "q"), q.dtype
    code = _args.dtype_code(q, "q")
    pq, sq = _args.heads(q, "q", dt, qs, dev)
    pk, sk = _args.heads(k, "k", dt, ks, dev)
    pwq, pwk = _args.need(w_q, "w_q", torch.float32, (d,), dev), _args.need(w_k, "w_k", torch.float32, (d,), dev)
    rot, pf, pp, pb = _rotation(inv_freq, positions, B, L, dev)
    made = []
    if out_q is None:
        out_q, poq, soq = _args.new_heads(qs, dt, dev, made)
    else:
        poq, soq = _args.heads_out(out_q, "out_q", dt, qs, dev)
    if out_k is None:
        out_k, pok, sok = _args.new_heads(ks, dt, dev, made)
    else:
        pok, sok = _args.heads_out(out_k, "out_k", dt, ks, dev)
    dm = _args.rope_dims(B, L, Hq, ks[1], d, rot, interleaved, norm, code, eps)
    _args.call(_native.lib.nats_qk_norm_rope, "nats_qk_norm_rope", dev, stream, made, dm, pq, sq, pk, sk, pwq, pwk, pf,
               pp, pb, _pos0(pos0), poq, soq, pok, sok)
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
    qs, ks = _pair(q, k)
    B, Hq, L, d = qs
    dev, dt, gt = _args.cuda_index(q, "q"), q.dtype, dq_out.dtype
    code = _args.dtype_code(q, "q")
    gcode = _args.dtype_code(dq_out, "dq_out")
    pq, sq = _args.heads(q, "q", dt, qs, dev)
    pk, sk = _args.heads(k, "k", dt, ks, dev)
    pgq, sgq = _args.heads(dq_out, "dq_out", gt, qs, dev)
    pgk, sgk = _args.heads(dk_out, "dk_out", gt, ks, dev)
    pwq, pwk = _args.need(w_q, "w_q", torch.float32, (d,), dev), _args.need(w_k, "w_k", torch.float32, (d,), dev)
    rot, pf, pp, pb = _rotation(inv_freq, positions, B, L, dev)
    made = []
    xt = dq.dtype if dq is not None else dk.dtype if dk is not None else dt
    if dq is None:
        dq, pdq, sdq = _args.new_heads(qs, xt, dev, made)
    else:
        pdq, sdq = _args.heads_out(dq, "dq", xt, qs, dev)
    if dk is None:
        dk, pdk, sdk = _args.new_heads(ks, xt, dev, made)
    else:
        pdk, sdk = _args.heads_out(dk, "dk", xt, ks, dev)
    xcode = _args.dtype_code(dq, "dq")
    dm = _args.rope_dims(B, L, Hq, ks[1], d, rot, interleaved, norm, code, eps)
    lib = _native.lib
    res = {"dq": dq, "dk": dk}
    pws, nws, pdw_q, pdw_k = None, 0, None, None
    if weight_grads and norm:
        res["dw_q"] = dw_q = torch.empty((d,), dtype=torch.float32, device=dev)
        res["dw_k"] = dw_k = torch.empty((d,), dtype=torch.float32, device=dev)
        pdw_q, pdw_k = dw_q.data_ptr(), dw_k.data_ptr()
        made += [dw_q, dw_k]
        if workspace is None:
            workspace = torch.empty(lib.nats_qk_norm_rope_bwd_workspace_size(dm), dtype=torch.uint8, device=dev)
            made.append(workspace)
        pws, nws = _args.need(workspace, "workspace", torch.uint8, None, dev), workspace.numel()
    _args.call(lib.nats_qk_norm_rope_bwd, "nats_qk_norm_rope_bwd", dev, stream, made, dm, gcode, xcode, pgq, sgq, pgk,
               sgk, pq, sq, pk, sk, pwq, pwk, pf, pp, pb, _pos0(pos0), pdq, sdq, pdk, sdk, pdw_q, pdw_k, pws, nws)
    return res
