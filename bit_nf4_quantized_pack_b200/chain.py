"""A chain of frozen-NF4 + LoRA layers with a saved-activation policy, and the
loss behind it.

A layer is a linear (``Layer``: Y_i = Y_{i-1} Ŵ_i + c_i (Y_{i-1} A_i) B_i) or a
gated block over two weights (``GatedLayer``: gate and up projections,
activation and product), as in a stack of a decoder layer's projections (its
attention and norms are not part of this library).  The backward walks the
layers in reverse.  What a layer keeps between the passes is the policy's:

    "save"       its input, and its rank-r products (a gated block: also g and u) in bf16
    "recompute"  its input alone; the backward forms the rest again, to the same bits
    "int8"       its input (a gated block: also g and u) as 8-bit checkpoints,
                 and its rank-r products in bf16

"recompute" keeps M·r bf16 less per linear, and 4·M·N bytes less per gated
block, at the price of a rank-r contraction, or the block's forward (the page
"SFT（四）：QLoRA的4-bit量化与LoRA微调原理", §26.2 为什么开启 Gradient Checkpointing,
states this trade); "int8" keeps 1.0625 bytes an element where "save" keeps 2,
and its gradients of A carry the checkpoint's rounding.

``HeadLoss`` is the softmax cross entropy behind an NF4 head;
``LinearChain.loss_backward`` runs a whole training step's passes through it.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass

import torch

from . import (_args, act8_quantize, gated_backward, gated_forward, head_loss_backward, head_loss_forward,
               linear_backward, linear_forward, new_status, status_sync)
from ._lib import QLoRAError

__all__ = ["Layer", "GatedLayer", "HeadLoss", "LinearChain"]

POLICIES = ("save", "recompute", "int8")


@dataclass
class Layer:
    w: object          # NF4Weight of the K_i x N_i frozen base
    A: torch.Tensor    # K_i x r bf16
    B: torch.Tensor    # r x N_i bf16
    c: float


@dataclass
class GatedLayer:
    """act(Y Ŵg + c (Y Ag) Bg) · (Y Ŵu + c (Y Au) Bu)."""
    wg: object         # NF4Weights of the K_i x N_i gate and up projections
    wu: object
    Ag: torch.Tensor   # K_i x r bf16
    Bg: torch.Tensor   # r x N_i bf16
    Au: torch.Tensor
    Bu: torch.Tensor
    c: float
    act: str = "silu"

    def args(self):
        return self.wg, self.wu, self.Ag, self.Bg, self.Au, self.Bu, self.c


def _on(t):
    """A context in which the tensor's device is current: the layer's calls and the
    status word's read-back take the current device and its stream."""
    return _args.on(t.device) if t.is_cuda else contextlib.nullcontext()


def _widths(layer):
    return (layer.wg if isinstance(layer, GatedLayer) else layer.w).shape


@dataclass
class HeadLoss:
    """Mean softmax cross entropy over the labels that are not ignore_index."""
    w: object                    # NF4Weight of the K x N head
    vocab: int | None = None     # columns that count (all N)
    ignore_index: int = -100

    def forward(self, X, labels, status=None):
        """Returns (mean loss, row losses, lse), all on the device."""
        loss, lse = head_loss_forward(X, self.w, labels, vocab=self.vocab, ignore_index=self.ignore_index,
                                      status=status)
        return loss.sum() / (labels != self.ignore_index).sum().clamp(min=1), loss, lse

    def backward(self, X, lse, labels, status=None):
        """dX of the mean loss."""
        counted = labels != self.ignore_index
        dloss = counted.to(torch.float32) / counted.sum().clamp(min=1)
        return head_loss_backward(dloss, X, lse, self.w, labels, vocab=self.vocab,
                                  ignore_index=self.ignore_index, status=status)


class LinearChain:
    def __init__(self, layers, policy: str = "save", head: HeadLoss | None = None):
        if policy not in POLICIES:
            raise ValueError("policy must be 'save', 'recompute' or 'int8'")
        for a, b in zip(layers, layers[1:]):
            if _widths(a)[1] != _widths(b)[0]:
                raise ValueError("layer widths do not chain")
        if head is not None and layers and _widths(layers[-1])[1] != head.w.shape[0]:
            raise ValueError("the head's width does not chain")
        self.layers = list(layers)
        self.policy = policy
        self.head = head
        self._inputs = None     # of the last forward
        self._zc = []

    def forward(self, X: torch.Tensor, status: torch.Tensor | None = None) -> torch.Tensor:
        with _on(X):
            own = status is None
            status = new_status(X.device) if own else status
            self._inputs, self._zc = [], []
            h = X
            for L in self.layers:
                self._inputs.append(act8_quantize(h, status=status) if self.policy == "int8" else h)
                if isinstance(L, GatedLayer):
                    save = {"save": "bf16", "int8": "int8", "recompute": None}[self.policy]
                    h, kept = gated_forward(h, *L.args(), act=L.act, save=save, status=status)
                else:
                    h, kept = linear_forward(h, L.w, L.A, L.B, L.c, status=status)
                self._zc.append(None if self.policy == "recompute" else kept)
            if own:
                self._check(status, "forward")
        return h

    def backward(self, dY: torch.Tensor, status: torch.Tensor | None = None):
        """Returns (dX, [the layers' adapter gradients]): (dA_i, dB_i) of a
        linear, (dAg_i, dBg_i, dAu_i, dBu_i) of a gated block."""
        if self._inputs is None:
            raise RuntimeError("backward before forward")
        with _on(dY):
            own = status is None
            status = new_status(dY.device) if own else status
            grads = [None] * len(self.layers)
            g = dY
            for i in reversed(range(len(self.layers))):
                L, x, kept = self.layers[i], self._inputs[i], self._zc[i]
                if isinstance(L, GatedLayer):
                    if kept is None:
                        _, kept = gated_forward(x, *L.args(), act=L.act, save="bf16", status=status)
                    g, *d = gated_backward(g, x, kept, *L.args(), act=L.act, status=status)
                else:
                    g, *d = linear_backward(g, x, kept, L.w, L.A, L.B, L.c, status=status)
                grads[i] = tuple(d)
            if own:
                self._check(status, "backward")
        return g, grads

    def loss_backward(self, X: torch.Tensor, labels: torch.Tensor, status: torch.Tensor | None = None):
        """The chain, its head's mean loss over `labels` (int64, one a row) and
        the backward through both.  Returns (mean loss, dX, adapter gradients)."""
        if self.head is None:
            raise RuntimeError("the chain has no head")
        with _on(X):
            own = status is None
            status = new_status(X.device) if own else status
            h = self.forward(X, status)
            mean, _, lse = self.head.forward(h, labels, status)
            dX, grads = self.backward(self.head.backward(h, lse, labels, status), status)
            if own:
                self._check(status, "loss_backward")
        return mean, dX, grads

    @staticmethod
    def _check(status, where):
        code, _ = status_sync(status)
        if code != 0:
            raise QLoRAError(code, f"LinearChain.{where}")
