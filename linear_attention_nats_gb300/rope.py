"""Query / key norm and rotation (nats_qk_norm_rope, nats_qk_norm_rope_bwd).

Operands are [B, H, L, d] views with any strides but the last, so q and k may
lie inside one projection's output, `qkv.view(B, L, 3, H, d)[:, :, 0].transpose(1, 2)`.
The checks of the arguments are in csrc/binding.cpp.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _native


def rope_inv_freq(rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """float64 [rot / 2]: base^(-2 i / rot), the radians per position of pair i."""
    return torch.tensor([float(base) ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=device)


def qk_norm_rope(q, k, w_q=None, w_k=None, inv_freq=None, positions=None, *, pos0: int = 0, interleaved: bool = False,
                 norm: bool = True, eps: float = 1e-6, out_q: Optional[torch.Tensor] = None,
                 out_k: Optional[torch.Tensor] = None, stream=None):
    """RMSNorm of every query and key row and its rotation, in one pass.

    q [B, Hq, L, d], k [B, Hk, L, d] bf16 or fp32 (d 64 or 128); w_q, w_k fp32
    [d] or None (unit); inv_freq float64 [rot / 2] (rope_inv_freq; None: no
    rotation; one that is not finite makes its pairs NaN); positions int64 [B, L] or [L], or None: pos0 + t; interleaved:
    pairs (2i, 2i + 1) in place of (i, i + rot / 2); norm=False rotates alone.
    Returns (q', k') in the layer's contiguous [B, H, L, d], or in out_q, out_k
    (any strides but the last; the inputs themselves for in place)."""
    return _native.operators.qk_norm_rope(q, k, w_q, w_k, inv_freq, positions, pos0, interleaved, norm, eps, out_q, out_k,
                                          stream)


def qk_norm_rope_bwd(dq_out, dk_out, q, k, w_q=None, w_k=None, inv_freq=None, positions=None, *, pos0: int = 0,
                     interleaved: bool = False, norm: bool = True, eps: float = 1e-6,
                     dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None, weight_grads: bool = True,
                     workspace=None, stream=None):
    """Gradient of qk_norm_rope: dq_out, dk_out (like its outputs; fp32, as
    hybrid_bwd gives them, or q's dtype) give a dict of dq, dk (q's dtype, or
    the given tensors' own: bf16 or fp32, any strides but the last) and, with
    weight_grads and norm, dw_q, dw_k (fp32 [d]).  q, k and the other arguments
    are the forward's."""
    return _native.operators.qk_norm_rope_bwd(dq_out, dk_out, q, k, w_q, w_k, inv_freq, positions, pos0, interleaved, norm,
                                              eps, dq, dk, weight_grads, workspace, stream)
