"""Argument checks shared by the operators' Python wrappers.

Each check raises before any device work: TypeError for a wrong type, dtype,
layout or device, ValueError for a wrong shape.  The library checks sizes it
can see (null pointers, alignment, supported shapes); what only the tensors
know, their extents, is checked here, so that a short buffer never reaches a
kernel.
"""
from __future__ import annotations

import contextlib

import torch

from ._lib import QLORA_DTYPE_BF16, QLORA_DTYPE_F32

GRAD_DTYPES = {torch.float32: QLORA_DTYPE_F32, torch.bfloat16: QLORA_DTYPE_BF16}

_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else None
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_here = contextlib.nullcontext()


def on(dev):
    """A context in which dev (a CUDA device with an index) is current; the
    usual case, that it is already, costs no switch."""
    if _current_device is not None and _current_device() == dev.index:
        return _here
    return torch.cuda.device(dev)


def stream(dev):
    """The raw current stream of dev."""
    if _raw_stream is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def cuda_2d(t, name):
    """A contiguous 2-D CUDA bf16 tensor; returns its shape and device."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA bfloat16 tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return t.shape[0], t.shape[1], t.device


def tensor(t, name, shape, dev, dtype=torch.bfloat16):
    """A contiguous tensor of `shape` and `dtype` on `dev`."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor on {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def weight(w, name, shape, dev):
    """An NF4Weight of `shape` whose buffers hold what its struct promises."""
    if tuple(w.shape) != shape:
        raise ValueError(f"{name} must be {shape[0]} x {shape[1]}, not {tuple(w.shape)}")
    numel = shape[0] * shape[1]
    n1 = (numel + 63) // 64
    _buffer(w.packed, torch.uint8, (numel + 1) // 2, name, dev)
    if w.double_quant:
        _buffer(w.code8, torch.uint8, n1, name, dev)
        _buffer(w.s2, torch.float32, (n1 + 255) // 256, name, dev)
        _buffer(w.offset, torch.float32, 1, name, dev)
    else:
        _buffer(w.absmax, torch.float32, n1, name, dev)


def _buffer(t, dtype, n, name, dev):
    if t is None or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        raise TypeError(f"{name}: a buffer is missing, or not a contiguous {dtype} tensor on {dev}")
    if t.numel() != n:
        raise ValueError(f"{name}: a buffer has {t.numel()} elements, not {n}")


def grad_code(dtype):
    if dtype not in GRAD_DTYPES:
        raise TypeError("grad_dtype must be torch.float32 or torch.bfloat16")
    return GRAD_DTYPES[dtype]


def ptr(t):
    return None if t is None else t.data_ptr()


def workspace(given, nbytes, dev):
    """The caller's workspace, or a new one from the caching allocator: it is
    ordered on the current stream, and under graph capture it belongs to that
    graph's own pool, so no two captured graphs or streams ever share one."""
    if given is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    if (not isinstance(given, torch.Tensor) or given.dtype != torch.uint8 or given.device != dev
            or not given.is_contiguous()):
        raise TypeError(f"workspace must be a contiguous uint8 tensor on {dev}")
    if given.numel() < nbytes:
        raise ValueError(f"workspace has {given.numel()} bytes, {nbytes} are needed")
    return given
