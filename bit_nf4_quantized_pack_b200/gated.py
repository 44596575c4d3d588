"""The gated feed-forward block over two NF4 frozen-base weights
(``qlora_gated_*`` in ``include/qlora_nf4.h``):

    g = X·Ŵg + c·(X·Ag)·Bg,   u = X·Ŵu + c·(X·Au)·Bu,   H = act(g)·u

and its backward.  The gate and up projections, the activation and the product
are one operation: g and u reach memory only where the backward needs them, in
bf16 or as 8-bit checkpoints.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

from . import _args
from ._lib import QLORA_ACT_GELU, QLORA_ACT_SILU, GatedSavedC, check, lib
from ._status import _finish, new_status
from .act8 import Act8, act8_struct, new_act8, width

__all__ = ["GatedSaved", "gated_forward", "gated_backward"]

ACTS = {"silu": QLORA_ACT_SILU, "gelu": QLORA_ACT_GELU}


@dataclass
class GatedSaved:
    """What the forward keeps for the backward: g and u (M x N, both bf16 or
    both ``Act8``) and the rank-r products Zg, Zu (M x r bf16)."""
    G: object
    U: object
    Zg: torch.Tensor
    Zu: torch.Tensor

    @staticmethod
    def empty(M: int, N: int, r: int, save: str, device="cuda") -> "GatedSaved":
        return _new_saved(M, N, r, save, torch.empty(0, dtype=torch.bfloat16, device=device))[0]

    def cstruct(self, M, N, r, dev) -> GatedSavedC:
        zg = _args.tensor(self.Zg, "saved.Zg", (M, r), dev)
        zu = _args.tensor(self.Zu, "saved.Zu", (M, r), dev)
        if isinstance(self.G, Act8):
            g, u = act8_struct(self.G, "saved.G", M, N, dev), act8_struct(self.U, "saved.U", M, N, dev)
            return GatedSavedC(None, None, g.codes, u.codes, g.scales, u.scales, zg, zu)
        return GatedSavedC(_args.tensor(self.G, "saved.G", (M, N), dev), _args.tensor(self.U, "saved.U", (M, N), dev),
                           None, None, None, None, zg, zu)


def _new_saved(M, N, r, save, like):
    """A new GatedSaved beside `like` (a bf16 tensor), and its C struct."""
    if save not in ("bf16", "int8"):
        raise ValueError("save must be None, 'bf16' or 'int8'")
    zg, zu = like.new_empty(M, r), like.new_empty(M, r)
    if save == "int8":
        (g, cg), (u, cu) = new_act8(M, N, like), new_act8(M, N, like)
        return GatedSaved(g, u, zg, zu), GatedSavedC(None, None, cg.codes, cu.codes, cg.scales, cu.scales,
                                                     zg.data_ptr(), zu.data_ptr())
    g, u = like.new_empty(M, N), like.new_empty(M, N)
    return GatedSaved(g, u, zg, zu), GatedSavedC(g.data_ptr(), u.data_ptr(), None, None, None, None, zg.data_ptr(),
                                                 zu.data_ptr())


def _kept(saved, M, N, r, dev):
    if not isinstance(saved, GatedSaved):
        raise TypeError("saved must be a GatedSaved")
    return saved.cstruct(M, N, r, dev)


def _act_code(act):
    if act not in ACTS:
        raise ValueError("act must be 'silu' or 'gelu'")
    return ACTS[act]


def _weights(K, dev, wg, wu, Ag, Bg, Au, Bu):
    """(N, r, the two weights' C structs, the four adapters' addresses)."""
    N = _args.columns(wg, "wg")
    if not isinstance(Ag, torch.Tensor) or Ag.dim() != 2:
        raise TypeError("Ag must be a matrix")
    r = Ag.shape[1]
    return (N, r, _args.weight(wg, "wg", K, N, dev), _args.weight(wu, "wu", K, N, dev),
            (_args.tensor(Ag, "Ag", (K, r), dev), _args.tensor(Bg, "Bg", (r, N), dev),
             _args.tensor(Au, "Au", (K, r), dev), _args.tensor(Bu, "Bu", (r, N), dev)))


def gated_forward(X, wg, wu, Ag, Bg, Au, Bu, c: float, *, act: str = "silu", save: str | None = None,
                  H=None, saved: GatedSaved | None = None, status=None, workspace=None):
    """H = act(X·Ŵg + c·(X·Ag)·Bg) · (X·Ŵu + c·(X·Au)·Bu); returns (H, saved).

    ``save`` None keeps nothing (inference; saved is None), "bf16" and "int8"
    return a ``GatedSaved`` for ``gated_backward``; ``saved`` gives the buffers
    it is written to instead.  wg and wu are K x N ``NF4Weight``s (either
    codebook, each with or without double quantization); Ag, Au K x r and Bg,
    Bu r x N bf16."""
    M, K, dev = _args.cuda_2d(X, "X")
    code = _act_code(act)
    N, r, cg, cu, adapters = _weights(K, dev, wg, wu, Ag, Bg, Au, Bu)
    with _args.on(dev):
        H = _args.output(H, X, "H", (M, N))
        kept = None
        if saved is not None:
            kept = _kept(saved, M, N, r, dev)
        elif save is not None:
            saved, kept = _new_saved(M, N, r, save, X)
        ws = _args.workspace(workspace, lib.qlora_gated_fwd_workspace_size(M, K, N, r), X)
        own = status is None
        status = new_status(dev) if own else status
        check(lib.qlora_gated_fwd(M, K, N, r, X.data_ptr(), C.byref(cg), C.byref(cu), *adapters, float(c), code,
                                  H.data_ptr(), C.byref(kept) if kept is not None else None, ws.data_ptr(), ws.numel(),
                                  _args.status(status, dev), _args.stream(dev)), "qlora_gated_fwd")
        if own:
            _finish(status, own, "qlora_gated_fwd")
    return H, saved


def gated_backward(dH, X, saved: GatedSaved, wg, wu, Ag, Bg, Au, Bu, c: float, *, act: str = "silu",
                   grad_dtype=torch.float32, dX=None, dAg=None, dBg=None, dAu=None, dBu=None, status=None,
                   workspace=None):
    """Returns (dX, dAg, dBg, dAu, dBu); X is the forward's input or its ``Act8``.
    The adapters' gradients are of ``grad_dtype`` (fp32 or bf16)."""
    M, N, dev = _args.cuda_2d(dH, "dH")
    code, gcode = _act_code(act), _args.grad_code(grad_dtype)
    is8 = isinstance(X, Act8)
    K = width(X, "X")
    x8 = act8_struct(X, "X", M, K, dev) if is8 else None
    x16 = None if is8 else _args.tensor(X, "X", (M, K), dev)
    Nw, r, cg, cu, adapters = _weights(K, dev, wg, wu, Ag, Bg, Au, Bu)
    if Nw != N:
        raise ValueError(f"dH must have {Nw} columns, not {N}")
    kept = _kept(saved, M, N, r, dev)
    with _args.on(dev):
        dX = _args.output(dX, dH, "dX", (M, K))
        dAg = _args.output(dAg, dH, "dAg", (K, r), grad_dtype)
        dBg = _args.output(dBg, dH, "dBg", (r, N), grad_dtype)
        dAu = _args.output(dAu, dH, "dAu", (K, r), grad_dtype)
        dBu = _args.output(dBu, dH, "dBu", (r, N), grad_dtype)
        ws = _args.workspace(workspace, lib.qlora_gated_bwd_workspace_size(M, K, N, r), dH)
        own = status is None
        status = new_status(dev) if own else status
        check(lib.qlora_gated_bwd(M, K, N, r, dH.data_ptr(), x16, C.byref(x8) if is8 else None, C.byref(kept),
                                  C.byref(cg), C.byref(cu), *adapters, float(c), code, dX.data_ptr(), dAg.data_ptr(),
                                  dBg.data_ptr(), dAu.data_ptr(), dBu.data_ptr(), gcode, ws.data_ptr(), ws.numel(),
                                  _args.status(status, dev), _args.stream(dev)), "qlora_gated_bwd")
        if own:
            _finish(status, own, "qlora_gated_bwd")
    return dX, dAg, dBg, dAu, dBu
