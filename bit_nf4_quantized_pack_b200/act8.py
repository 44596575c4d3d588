"""8-bit activation checkpoints (``qlora_act8_*`` in ``include/qlora_nf4.h``).

A bf16 matrix that a layer keeps between its forward and its backward, in int8
codes with one fp32 scale per 64 consecutive elements of a row: 1.0625 bytes an
element instead of 2.  ``linear_backward`` and ``gated_backward`` take an
``Act8`` in the place of their input and read the codes directly;
``LinearChain(policy="int8")`` keeps every layer's input this way.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

from . import _args
from ._lib import Act8C, check, lib
from ._status import _finish, new_status

__all__ = ["Act8", "act8_quantize", "act8_dequantize"]


@dataclass
class Act8:
    """The checkpoint of an M x K matrix: ``codes`` int8 M x K and ``scales``
    fp32 M x (K / 64)."""
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device

    @staticmethod
    def empty(rows: int, cols: int, device="cuda") -> "Act8":
        return Act8(torch.empty((rows, cols), dtype=torch.int8, device=device),
                    torch.empty((rows, cols // 64), dtype=torch.float32, device=device))


def act8_struct(a, name, M, K, dev):
    """The C struct of an Act8 of M x K on `dev` with buffers of the right extents."""
    if not isinstance(a, Act8):
        raise TypeError(f"{name} must be an Act8")
    return Act8C(M, K, _args.tensor(a.codes, name, (M, K), dev, torch.int8),
                 _args.tensor(a.scales, name, (M, K // 64), dev, torch.float32))


def width(X, name):
    """The columns of a matrix or of an Act8 (-1 where it has not two dimensions)."""
    t = X.codes if isinstance(X, Act8) else X
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a matrix or its Act8")
    return t.shape[1] if t.dim() == 2 else -1


def new_act8(M, K, like):
    """A new Act8 of M x K beside `like`, and its C struct."""
    codes = like.new_empty(M, K, dtype=torch.int8)
    scales = like.new_empty(M, K // 64, dtype=torch.float32)
    return Act8(codes, scales), Act8C(M, K, codes.data_ptr(), scales.data_ptr())


def act8_quantize(X: torch.Tensor, *, out: Act8 | None = None, status: torch.Tensor | None = None) -> Act8:
    """The 8-bit checkpoint of a contiguous CUDA bf16 matrix whose row length
    is a multiple of 64.  A NaN or infinity in X is a device error."""
    M, K, dev = _args.cuda_2d(X, "X")
    with _args.on(dev):
        if out is None:
            out, st = new_act8(M, K, X)
        else:
            st = act8_struct(out, "out", M, K, dev)
        own = status is None
        status = new_status(dev) if own else status
        check(lib.qlora_act8_quantize(X.data_ptr(), C.byref(st), _args.status(status, dev), _args.stream(dev)),
              "qlora_act8_quantize")
        if own:
            _finish(status, own, "qlora_act8_quantize")
    return out


def act8_dequantize(a: Act8, *, out: torch.Tensor | None = None) -> torch.Tensor:
    """The bf16 matrix that the checkpoint stands for."""
    if (not isinstance(a, Act8) or not isinstance(a.codes, torch.Tensor) or not a.codes.is_cuda
            or a.codes.dim() != 2):
        raise TypeError("a must be an Act8 on a CUDA device")
    M, K = a.codes.shape
    dev = a.device
    st = act8_struct(a, "a", M, K, dev)
    with _args.on(dev):
        out = _args.output(out, a.codes, "out", (M, K))
        check(lib.qlora_act8_dequantize(C.byref(st), out.data_ptr(), _args.stream(dev)), "qlora_act8_dequantize")
    return out
