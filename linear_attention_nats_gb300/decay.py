"""Linear attention with a decay for each head (nats_decay_attn,
nats_decay_attn_bwd, nats_decay_attn_step): S_t = e^g S_(t-1) + v_t k_t^T,
o_t = scale S_t q_t, over a prompt, its gradient, and one new token.

Operands are [B, H, L, d] views with any strides but the last, so q, k and v
may lie inside one projection's output, `qkv.view(B, L, 3, H, d)[:, :, 0].transpose(1, 2)`.
States are fp32 [B, H, d, d], a value's entries as rows.  The checks of the
arguments are in csrc/binding.cpp.

bf16 operands go to the tensor cores where every row starts at a multiple of 16
bytes and no dimension is expanded; others take the fp32 kernel, which is 5 to 20
times slower, so that a contiguous copy of them first is cheaper.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _native


def decay_attn(q, k, v, log_decay, *, scale: float = 0.0, lens=None, state=None, return_state: bool = False,
               state_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, workspace=None, stream=None):
    """Linear attention over a prompt: q, k, v [B, H, L, d] bf16 or fp32 (d 64
    or 128, any L); log_decay fp32 [H] (the log of each head's decay, <= 0, a
    constant without gradient); scale 0 for 1 / sqrt(d); lens int32 [B]
    or None: the tokens of each sequence, those behind them take no part and
    their rows of the output are zero; state: the one ahead of the first
    token (None: zero).  Returns out (contiguous, or the given tensor, which
    must not share memory with q, k or v), or (out, the state after the last
    token) with return_state or state_out, which may be `state` itself."""
    return _native.operators.decay_attn(q, k, v, log_decay, scale, lens, state, return_state, state_out, out, workspace,
                                        stream)


def decay_attn_bwd(dout, q, k, v, log_decay, *, scale: float = 0.0, lens=None, state=None, dstate_out=None,
                   state_grad: bool = False, dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                   dv: Optional[torch.Tensor] = None, workspace=None, stream=None):
    """Gradient of decay_attn: dout, the gradient of its output (q's type), and
    dstate_out, that of its last state (fp32, or None: zero), give a dict of
    dq, dk, dv (q's type, contiguous or the given tensors, which must not share
    memory with an input or one another) and, with state_grad, dstate, the
    gradient of `state` (fp32).  The other arguments are the forward's.  Rows
    behind a sequence's end are zero."""
    return _native.operators.decay_attn_bwd(dout, q, k, v, log_decay, scale, lens, state, dstate_out, state_grad, dq, dk, dv,
                                            workspace, stream)


def decay_attn_step(q, k, v, log_decay, state, *, scale: float = 0.0, out: Optional[torch.Tensor] = None, stream=None):
    """One new token of each sequence: q, k, v [B, H, d] (any strides but the
    last) on `state`, fp32 [B, H, d, d], which is updated in place.  Returns
    out [B, H, d] (contiguous, or the given tensor, which must not share memory
    with q, k or v)."""
    return _native.operators.decay_attn_step(q, k, v, log_decay, state, scale, out, stream)


def decay_attn_check(stream=None) -> None:
    """Synchronises with `stream` (None: the current one) and raises NatsError
    if a kernel of decay_attn or decay_attn_bwd has given up on a bounded wait
    on that stream's device since the last such report."""
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        _native.check(_native.lib.nats_decay_attn_check(s.cuda_stream), "nats_decay_attn_check")
