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

from ._lib import QLORA_DTYPE_BF16, QLORA_DTYPE_F32, NF4StateC

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
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA bfloat16 tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions")
    return shape[0], shape[1], t.device


def tensor(t, name, shape, dev, dtype=torch.bfloat16):
    """The address of a contiguous tensor of `shape` and `dtype` on `dev`."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor on {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr()


def columns(w, name):
    """The columns of an NF4Weight (-1 where it has not two dimensions)."""
    if not hasattr(w, "packed"):
        raise TypeError(f"{name} must be an NF4Weight")
    shape = w.shape
    return shape[1] if len(shape) == 2 else -1


def weight(w, name, K, N, dev):
    """The C struct of an NF4Weight of K x N whose buffers hold what it promises."""
    if not hasattr(w, "packed"):
        raise TypeError(f"{name} must be an NF4Weight")
    shape = w.shape
    if len(shape) != 2 or shape[0] != K or shape[1] != N:
        raise ValueError(f"{name} must be {K} x {N}, not {tuple(shape)}")
    numel = K * N
    n1 = (numel + 63) // 64
    packed = _buffer(w.packed, torch.uint8, (numel + 1) // 2, name, dev)
    if w.double_quant:
        return NF4StateC(numel, 64, 1, 256, w.codebook, packed, None, _buffer(w.code8, torch.uint8, n1, name, dev),
                         _buffer(w.s2, torch.float32, (n1 + 255) // 256, name, dev),
                         _buffer(w.offset, torch.float32, 1, name, dev))
    return NF4StateC(numel, 64, 0, 256, w.codebook, packed, _buffer(w.absmax, torch.float32, n1, name, dev))


def _buffer(t, dtype, n, name, dev):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        raise TypeError(f"{name}: a buffer is missing, or not a contiguous {dtype} tensor on {dev}")
    if t.numel() != n:
        raise ValueError(f"{name}: a buffer has {t.numel()} elements, not {n}")
    return t.data_ptr()


def output(t, like, name, shape, dtype=torch.bfloat16):
    """`t` checked, or a new tensor of `shape` and `dtype` beside `like`."""
    if t is None:
        return like.new_empty(*shape, dtype=dtype)   # (a size as one tuple costs half as much again)
    tensor(t, name, shape, like.device, dtype)
    return t


def grad_code(dtype):
    if dtype not in GRAD_DTYPES:
        raise TypeError("grad_dtype must be torch.float32 or torch.bfloat16")
    return GRAD_DTYPES[dtype]


def status(given, dev):
    """The address of the caller's status word."""
    if (not isinstance(given, torch.Tensor) or given.dtype is not torch.int32 or given.device != dev
            or given.numel() < 1):
        raise TypeError(f"status must be an int32 tensor on {dev} (see new_status)")
    return given.data_ptr()


def workspace(given, nbytes, like):
    """The caller's workspace, or a new one from the caching allocator: it is
    ordered on the current stream, and under graph capture it belongs to that
    graph's own pool, so no two captured graphs or streams ever share one."""
    if given is None:
        return like.new_empty(max(nbytes, 256), dtype=torch.uint8)
    dev = like.device
    if (not isinstance(given, torch.Tensor) or given.dtype != torch.uint8 or given.device != dev
            or not given.is_contiguous()):
        raise TypeError(f"workspace must be a contiguous uint8 tensor on {dev}")
    if given.numel() < nbytes:
        raise ValueError(f"workspace has {given.numel()} bytes, {nbytes} are needed")
    return given
