"""8-bit activation checkpoints — CPU oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The codec is defined in fp32 steps: blocks of 64 along a row, scale
s = fl32(amax / 127) (1 below the normal range), code = rint(fl32(x / s)) with
ties to even, value = bf16(fl32(code * s)).  NumPy's float32 divide and
multiply round once each, as the definition asks.
"""
from __future__ import annotations

import numpy as np

from .nf4 import round_to_bf16


def act8_quantize(X):
    """(codes int8 M x K, scales fp32 M x K/64) of a bf16-valued matrix."""
    X = np.asarray(X, dtype=np.float32)
    M, K = X.shape
    blocks = X.reshape(M, K // 64, 64)
    s = np.max(np.abs(blocks), axis=2) / np.float32(127)
    s = np.where(s >= np.finfo(np.float32).tiny, s, np.float32(1)).astype(np.float32)
    q = np.rint(blocks / s[:, :, None])
    return q.astype(np.int8).reshape(M, K), s


def act8_dequantize(codes, scales):
    """The bf16 values the codes stand for, in fp64."""
    M, K = codes.shape
    v = codes.astype(np.float32).reshape(M, K // 64, 64) * scales[:, :, None]
    return np.asarray(round_to_bf16(v.astype(np.float64)), dtype=np.float64).reshape(M, K)
