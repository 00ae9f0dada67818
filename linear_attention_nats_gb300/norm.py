"""Layer norm and its gradient (nats_layer_norm, nats_layer_norm_bwd).

Rows are the last dimension of tensors of any shape; the dimensions ahead of
it may lie in any order in memory, so a norm of each head's output takes a
view of [B, L, H, d] as it is.  The checks of the arguments are in
csrc/binding.cpp.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _native


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-6, out: Optional[torch.Tensor] = None, stream=None):
    """Layer norm of the rows of x [..., D], bf16 or fp32, D from 1 to 16384:
    (x - mean) / sqrt(var + eps) * weight + bias, weight and bias fp32 [D] or
    None (1 and 0).  Any strides but the last; the dimensions ahead of it must
    come down to three where neighbours that follow one another in memory are
    one.  Returns a new contiguous tensor, or out (x itself for in place; no
    other memory of x)."""
    return _native.operators.layer_norm(x, weight, bias, eps, out, stream)


def layer_norm_bwd(dout, x, weight=None, *, eps: float = 1e-6, dx: Optional[torch.Tensor] = None,
                   weight_grads: bool = True, workspace=None, stream=None):
    """Gradient of layer_norm: dout (x's type and shape) and the forward's x,
    weight and eps give a dict of dx (x's type; the given tensor, which may be
    dout or x itself, but no other memory of theirs) and, with weight_grads, dw
    and db (fp32 [D], the gradients of weight and bias)."""
    return _native.operators.layer_norm_bwd(dout, x, weight, eps, dx, weight_grads, workspace, stream)
