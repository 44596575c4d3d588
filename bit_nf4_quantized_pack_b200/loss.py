"""Softmax cross entropy behind an NF4 frozen head, the logits never in memory
(``qlora_head_loss_*`` in ``include/qlora_nf4.h``):

    l = X·Ŵ,  lse = log Σ exp(l),  loss = lse - l[label]
    dX = dloss · (softmax(l) - onehot(label)) · Ŵᵀ
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _args
from ._lib import check, lib
from ._status import _finish, new_status

__all__ = ["head_loss_forward", "head_loss_backward"]


def _head(X, w, labels, vocab):
    M, K, dev = _args.cuda_2d(X, "X")
    N = _args.columns(w, "w")
    st = _args.weight(w, "w", K, N, dev)
    y = _args.tensor(labels, "labels", (M,), dev, torch.int64)
    vocab = N if vocab is None else int(vocab)
    if not 1 <= vocab <= N:
        raise ValueError(f"vocab must be 1 .. {N}, not {vocab}")
    return M, K, N, vocab, dev, st, y


def head_loss_forward(X, w, labels, *, vocab: int | None = None, ignore_index: int = -100, loss=None,
                      lse=None, status=None, workspace=None):
    """Per-row losses and log-sum-exps (fp32, M each) of the logits X·Ŵ.

    w is the K x N ``NF4Weight`` of the head; its columns from ``vocab`` on (all
    N by default) are padding.  Rows whose label is ``ignore_index`` have loss
    0; any other label outside 0 .. vocab - 1 is a device error."""
    M, K, N, vocab, dev, st, y = _head(X, w, labels, vocab)
    with _args.on(dev):
        loss = _args.output(loss, X, "loss", (M,), torch.float32)
        lse = _args.output(lse, X, "lse", (M,), torch.float32)
        ws = _args.workspace(workspace, lib.qlora_head_loss_fwd_workspace_size(M, K, N), X)
        own = status is None
        status = new_status(dev) if own else status
        check(lib.qlora_head_loss_fwd(M, K, N, vocab, X.data_ptr(), C.byref(st), y, int(ignore_index),
                                      loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
                                      _args.status(status, dev), _args.stream(dev)), "qlora_head_loss_fwd")
        if own:
            _finish(status, own, "qlora_head_loss_fwd")
    return loss, lse


def head_loss_backward(dloss, X, lse, w, labels, *, vocab: int | None = None, ignore_index: int = -100,
                       dX=None, status=None, workspace=None):
    """dX (bf16 M x K) from dloss (fp32 M, the gradient of each row's loss: 1/count
    for the mean over count labels) and the forward's lse."""
    M, K, N, vocab, dev, st, y = _head(X, w, labels, vocab)
    dl = _args.tensor(dloss, "dloss", (M,), dev, torch.float32)
    ls = _args.tensor(lse, "lse", (M,), dev, torch.float32)
    with _args.on(dev):
        dX = _args.output(dX, X, "dX", (M, K))
        ws = _args.workspace(workspace, lib.qlora_head_loss_bwd_workspace_size(M, K, N), X)
        own = status is None
        status = new_status(dev) if own else status
        check(lib.qlora_head_loss_bwd(M, K, N, vocab, dl, X.data_ptr(), ls, C.byref(st), y, int(ignore_index),
                                      dX.data_ptr(), ws.data_ptr(), ws.numel(), _args.status(status, dev),
                                      _args.stream(dev)), "qlora_head_loss_bwd")
        if own:
            _finish(status, own, "qlora_head_loss_bwd")
    return dX
