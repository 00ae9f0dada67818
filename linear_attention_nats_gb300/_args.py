"""Argument checks and the call itself, shared by the operator modules.

A small call's time is this file's: each check is one comparison on the way
through, and what explains a refusal is worked out only once one has failed."""

from __future__ import annotations

from functools import lru_cache

import torch

from . import _native
from ._native import NATS_BF16, NATS_F32, RopeDims, Strides

_CODES = {torch.bfloat16: NATS_BF16, torch.float32: NATS_F32}
_raw_stream = torch._C._cuda_getCurrentRawStream

# the C structs of sizes and strides, by their values (never written after)
strides = lru_cache(maxsize=4096)(Strides)
rope_dims = lru_cache(maxsize=4096)(RopeDims)


def dtype_code(t: torch.Tensor, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def cuda_index(t: torch.Tensor, name: str) -> int:
    """The index of the tensor's CUDA device."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def refuse(t, name, dtype, shape, dev):
    """Raises what is wrong with a tensor argument that has failed a check."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def int32(**values):
    """Refuses integers that a 32-bit argument would cut off."""
    for name, v in values.items():
        if not -(1 << 31) <= v < 1 << 31:
            raise ValueError(f"{name} = {v} does not fit 32 bits")


def need(t, name, dtype, shape, dev):
    """The address of a contiguous tensor argument on device `dev` (None for None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and (shape is None or t.shape == shape) and t.is_contiguous():
        return t.data_ptr()
    refuse(t, name, dtype, shape, dev)


def heads(t, name, dtype, shape, dev):
    """A [B, H, L, d] operand with any strides but the last: its address and strides."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        refuse(t, name, dtype, shape, dev)
    b, h, s, e = t.stride()
    if e != 1 and t.numel() > 0:
        raise ValueError(f"{name}: the entries of a row must be contiguous (last stride 1, got {e})")
    return t.data_ptr(), strides(b, h, s)


def heads_out(t, name, dtype, shape, dev):
    """The same for an output, which must not be an expanded tensor (entries that share an address)."""
    p, st = heads(t, name, dtype, shape, dev)
    if not (st.b and st.h and st.t):
        for n, s in zip(t.shape, t.stride()):
            if s == 0 and n > 1:
                raise ValueError(f"{name} is written and must not be an expanded tensor")
    return p, st


def new_heads(shape, dtype, dev, made):
    """A new contiguous [B, H, L, d] output (added to `made`), its address and strides."""
    t = torch.empty(shape, dtype=dtype, device=dev)
    made.append(t)
    _, h, s, e = shape
    return t, t.data_ptr(), strides(h * s * e, s * e, e)


def call(fn, where, dev, stream, made, *args):
    """fn(*args, stream) on device `dev`.  `made`: tensors allocated for the
    call (on the current stream), which a call on another stream keeps alive
    until it has run."""
    handle = _raw_stream(dev)
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
        if stream.cuda_stream != handle:
            handle = stream.cuda_stream
            for t in made:
                t.record_stream(stream)
    if dev == torch._C._cuda_getDevice():
        code = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, handle)
    if code:
        raise _native.NatsError(code, where)
