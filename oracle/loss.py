"""Softmax cross entropy behind a frozen head — CPU oracle (fp64).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

    l = X W[:, :vocab],  lse = log sum exp l,  loss = lse - l[label]
    dX = dloss (softmax(l) - onehot(label)) W[:, :vocab]^T
Rows whose label is ignore_index have loss 0 and no gradient.  Pinned by
central differences of ``head_loss_forward``.
"""
from __future__ import annotations

import numpy as np


def head_loss_forward(X, W, labels, vocab, ignore_index=-100):
    """Returns (loss, lse)."""
    logits = np.asarray(X, dtype=np.float64) @ np.asarray(W, dtype=np.float64)[:, :vocab]
    top = logits.max(axis=1)
    lse = np.log(np.exp(logits - top[:, None]).sum(axis=1)) + top
    loss = np.zeros(len(labels))
    for i, y in enumerate(labels):
        if y != ignore_index:
            loss[i] = lse[i] - logits[i, y]
    return loss, lse


def head_loss_backward(dloss, X, W, labels, vocab, ignore_index=-100):
    """Returns dX."""
    W = np.asarray(W, dtype=np.float64)[:, :vocab]
    logits = np.asarray(X, dtype=np.float64) @ W
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    for i, y in enumerate(labels):
        if y == ignore_index:
            p[i] = 0
        else:
            p[i, y] -= 1
            p[i] *= dloss[i]
    return p @ W.T
