"""The device status word: errors that only the device can see accumulate in it
(see ``include/qlora_nf4.h``)."""
from __future__ import annotations

import ctypes as C

import torch

from ._lib import check, lib


def _stream():
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return C.c_void_p(t.data_ptr()) if t is not None else C.c_void_p(0)


def new_status(device="cuda") -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def status_sync(status: torch.Tensor):
    """(first error code or 0, raw bit mask); synchronizes the current stream."""
    mask = C.c_int32(0)
    code = lib.qlora_status_sync(_ptr(status), _stream(), C.byref(mask))
    return int(code), int(mask.value)


def status_clear(status: torch.Tensor) -> None:
    check(lib.qlora_status_clear(_ptr(status), _stream()), "qlora_status_clear")


def _finish(status, own_status, where):
    if own_status:
        code, _ = status_sync(status)
        check(code, where)
