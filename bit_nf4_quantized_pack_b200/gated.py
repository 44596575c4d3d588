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
from .act8 import Act8, check_act8

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
        def pre():
            if save == "int8":
                return Act8.empty(M, N, device)
            return torch.empty((M, N), dtype=torch.bfloat16, device=device)

        def z():
            return torch.empty((M, r), dtype=torch.bfloat16, device=device)
        if save not in ("bf16", "int8"):
            raise ValueError("save must be 'bf16' or 'int8'")
        return GatedSaved(pre(), pre(), z(), z())

    def cstruct(self, M, N, r, dev) -> GatedSavedC:
        _args.tensor(self.Zg, "saved.Zg", (M, r), dev)
        _args.tensor(self.Zu, "saved.Zu", (M, r), dev)
        s = GatedSavedC(Zg=self.Zg.data_ptr(), Zu=self.Zu.data_ptr())
        if isinstance(self.G, Act8):
            check_act8(self.G, "saved.G", (M, N), dev)
            check_act8(self.U, "saved.U", (M, N), dev)
            s.G8, s.G_scales = self.G.codes.data_ptr(), self.G.scales.data_ptr()
            s.U8, s.U_scales = self.U.codes.data_ptr(), self.U.scales.data_ptr()
        else:
            _args.tensor(self.G, "saved.G", (M, N), dev)
            _args.tensor(self.U, "saved.U", (M, N), dev)
            s.G, s.U = self.G.data_ptr(), self.U.data_ptr()
        return s


def _act_code(act):
    if act not in ACTS:
        raise ValueError("act must be 'silu' or 'gelu'")
    return ACTS[act]


def _weights(K, dev, wg, wu, Ag, Bg, Au, Bu):
    N = wg.shape[1] if len(wg.shape) == 2 else -1
    _args.weight(wg, "wg", (K, N), dev)
    _args.weight(wu, "wu", (K, N), dev)
    if not isinstance(Ag, torch.Tensor) or Ag.dim() != 2:
        raise TypeError("Ag must be a matrix")
    r = Ag.shape[1]
    for t, name, shape in ((Ag, "Ag", (K, r)), (Bg, "Bg", (r, N)), (Au, "Au", (K, r)), (Bu, "Bu", (r, N))):
        _args.tensor(t, name, shape, dev)
    return N, r


def gated_forward(X, wg, wu, Ag, Bg, Au, Bu, c: float, *, act: str = "silu", save: str | None = None,
                  H=None, saved: GatedSaved | None = None, status=None, workspace=None):
    """H = act(X·Ŵg + c·(X·Ag)·Bg) · (X·Ŵu + c·(X·Au)·Bu); returns (H, saved).

    ``save`` None keeps nothing (inference; saved is None), "bf16" and "int8"
    return a ``GatedSaved`` for ``gated_backward``; ``saved`` gives the buffers
    it is written to instead.  wg and wu are K x N ``NF4Weight``s (either
    codebook, each with or without double quantization); Ag, Au K x r and Bg,
    Bu r x N bf16."""
    from . import _finish, new_status
    M, K, dev = _args.cuda_2d(X, "X")
    code = _act_code(act)
    N, r = _weights(K, dev, wg, wu, Ag, Bg, Au, Bu)
    with _args.on(dev):
        if H is None:
            H = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        else:
            _args.tensor(H, "H", (M, N), dev)
        if saved is None and save is not None:
            saved = GatedSaved.empty(M, N, r, save, dev)
        kept = C.byref(saved.cstruct(M, N, r, dev)) if saved is not None else None
        need = lib.qlora_gated_fwd_workspace_size(M, K, N, r)
        ws = _args.workspace(workspace, need, dev)
        own = status is None
        status = new_status(dev) if own else status
        check(lib.qlora_gated_fwd(M, K, N, r, X.data_ptr(), C.byref(wg.cstruct()), C.byref(wu.cstruct()),
                                  Ag.data_ptr(), Bg.data_ptr(), Au.data_ptr(), Bu.data_ptr(), float(c), code,
                                  H.data_ptr(), kept, ws.data_ptr(), ws.numel(), status.data_ptr(),
                                  _args.stream(dev)), "qlora_gated_fwd")
        _finish(status, own, "qlora_gated_fwd")
    return H, saved


def gated_backward(dH, X, saved: GatedSaved, wg, wu, Ag, Bg, Au, Bu, c: float, *, act: str = "silu",
                   grad_dtype=torch.float32, dX=None, dAg=None, dBg=None, dAu=None, dBu=None, status=None,
                   workspace=None):
    """Returns (dX, dAg, dBg, dAu, dBu); X is the forward's input or its ``Act8``.
    The adapters' gradients are of ``grad_dtype`` (fp32 or bf16)."""
    from . import _finish, new_status
    M, N, dev = _args.cuda_2d(dH, "dH")
    code, gcode = _act_code(act), _args.grad_code(grad_dtype)
    is8 = isinstance(X, Act8)
    K = X.shape[1] if (is8 or isinstance(X, torch.Tensor)) and len(X.shape) == 2 else -1
    if is8:
        check_act8(X, "X", (M, K), dev)
    else:
        _args.tensor(X, "X", (M, K), dev)
    Nw, r = _weights(K, dev, wg, wu, Ag, Bg, Au, Bu)
    if Nw != N:
        raise ValueError(f"dH must have {Nw} columns, not {N}")
    if not isinstance(saved, GatedSaved):
        raise TypeError("saved must be the GatedSaved of the forward")
    with _args.on(dev):
        kept = saved.cstruct(M, N, r, dev)
        out = []
        for t, name, shape, dt in ((dX, "dX", (M, K), torch.bfloat16), (dAg, "dAg", (K, r), grad_dtype),
                                   (dBg, "dBg", (r, N), grad_dtype), (dAu, "dAu", (K, r), grad_dtype),
                                   (dBu, "dBu", (r, N), grad_dtype)):
            if t is None:
                t = torch.empty(shape, dtype=dt, device=dev)
            else:
                _args.tensor(t, name, shape, dev, dt)
            out.append(t)
        need = lib.qlora_gated_bwd_workspace_size(M, K, N, r)
        ws = _args.workspace(workspace, need, dev)
        own = status is None
        status = new_status(dev) if own else status
        x8 = C.byref(X.cstruct()) if is8 else None
        check(lib.qlora_gated_bwd(M, K, N, r, dH.data_ptr(), None if is8 else X.data_ptr(), x8,
                                  C.byref(kept), C.byref(wg.cstruct()), C.byref(wu.cstruct()),
                                  Ag.data_ptr(), Bg.data_ptr(), Au.data_ptr(), Bu.data_ptr(), float(c), code,
                                  *(t.data_ptr() for t in out), gcode, ws.data_ptr(), ws.numel(),
                                  status.data_ptr(), _args.stream(dev)), "qlora_gated_bwd")
        _finish(status, own, "qlora_gated_bwd")
    return tuple(out)
