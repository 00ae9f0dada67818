"""Argument checks shared by the operator modules: tensors of one device, and
the stream that a call runs on."""

from __future__ import annotations

import contextlib

import torch

from ._native import NATS_BF16, NATS_F32, Strides

_CODES = {torch.bfloat16: NATS_BF16, torch.float32: NATS_F32}


def dtype_code(t: torch.Tensor, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def need(t, name, dtype=None, shape=None, device=None, contiguous=True):
    """Checks one tensor argument and returns its address (None for None)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def heads(t, name, dtype, shape, device):
    """A [B, H, L, d] operand with any strides but the last: its address and strides."""
    p = need(t, name, dtype, shape, device, contiguous=False)
    b, h, t_, e = t.stride()
    if e != 1 and t.shape[3] > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the entries of a row must be contiguous (last stride 1, got {e})")
    return p, Strides(b, h, t_)


def distinct(t, name):
    """Refuses an output some of whose elements share an address (an expanded tensor)."""
    for n, s in zip(t.shape, t.stride()):
        if s == 0 and n > 1:
            raise ValueError(f"{name} is written and must not be an expanded tensor")


@contextlib.contextmanager
def launch(device, stream, made=()):
    """The handle of the stream a call runs on, with `device` the current one.
    `made`: tensors allocated for the call (on the current stream), which a
    call on another stream keeps alive until it has run."""
    cur = torch.cuda.current_stream(device)
    s = cur if stream is None else stream
    if s.device != device:
        raise ValueError(f"the stream is on {s.device}, the tensors on {device}")
    if s != cur:
        for t in made:
            if t is not None:
                t.record_stream(s)
    if device.index == torch.cuda.current_device():
        yield s.cuda_stream
    else:
        with torch.cuda.device(device):
            yield s.cuda_stream


def workspace(given, size, device):
    """The caller's workspace, or a new one (second value: whether it is new), its address and its bytes."""
    if given is None:
        w = torch.empty(max(size, 1), dtype=torch.uint8, device=device)
        return w, True
    need(given, "workspace", torch.uint8, None, device)
    return given, False
