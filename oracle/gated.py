"""Gated feed-forward block over two frozen-base LoRA layers — CPU oracle (fp64).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

    g = X Wg + c (X Ag) Bg,  u = X Wu + c (X Au) Bu,  H = act(g) u
    dg = dH u act'(g),  du = dH act(g),  and for each of the two layers the
    backward of ``oracle.linear.lora_backward``; dX is the sum of both.
Pinned by central differences of ``gated_forward``.
"""
from __future__ import annotations

import numpy as np

from .linear import lora_backward, lora_forward


def act(g, kind):
    """(act(g), act'(g)) in fp64."""
    g = np.asarray(g, dtype=np.float64)
    if kind == "silu":
        s = 0.5 * (1 + np.tanh(0.5 * g))
        return g * s, s + g * s * (1 - s)
    k = np.sqrt(2 / np.pi)
    t = np.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def gated_forward(X, Wg, Wu, Ag, Bg, Au, Bu, c, kind):
    """Returns (H, g, u, Zg, Zu) with Z = c X A."""
    g, Zg = lora_forward(X, Wg, Ag, Bg, c)
    u, Zu = lora_forward(X, Wu, Au, Bu, c)
    return act(g, kind)[0] * u, g, u, c * Zg, c * Zu


def gated_pre_grads(dH, g, u, kind):
    """(dg, du)."""
    a, d = act(g, kind)
    dH = np.asarray(dH, dtype=np.float64)
    return dH * u * d, dH * a


def gated_backward(dH, X, g, u, Wg, Wu, Ag, Bg, Au, Bu, c, kind):
    """Returns (dX, dAg, dBg, dAu, dBu)."""
    dg, du = gated_pre_grads(dH, g, u, kind)
    dXg, dAg, dBg = lora_backward(dg, X, Wg, Ag, Bg, c)
    dXu, dAu, dBu = lora_backward(du, X, Wu, Au, Bu, c)
    return dXg + dXu, dAg, dBg, dAu, dBu
