"""Error bounds of the gated block, the 8-bit checkpoints and the head loss,
and the inputs of their GPU tests.

The bounds are element by element and follow the operators' own roundings:

* a rounding to bf16 is off by at most half a step, 2^-8 of the value (HALF);
* a sum of n products in fp32 is off by at most n 2^-23 of the sum of the
  products' magnitudes (each of its n additions rounds, or truncates, once;
  the products of bf16 operands are exact);
* the activation functions go through the hardware's base-2 exponential and a
  fast division: 2^-18 of the value covers both (a few units of 2^-22 each).

Products of two errors are covered by the factor 1.01 on the total.
"""
import numpy as np

from inputs import synthetic as S
from oracle import int4, nf4
from oracle.gated import act
from tests._gpu_util import OracleWeight, assert_close, to_dev, to_np  # noqa: F401

HALF = 2.0 ** -8
FAST = 2.0 ** -18
TINY = 1e-30
SLACK = 1.01


def gamma(n):
    return n * 2.0 ** -23


class DecodedWeight:
    """A quantized weight on the device, and the operand its kernels decode:
    bf16(fl32(code value * scale)) from the oracle's codes and scales."""

    def __init__(self, W, kind):
        import bit_nf4_quantized_pack_b200 as q
        K, N = W.shape
        if kind == "int4":
            self.dev = q.quantize(to_dev(W), codebook="int4")
            codes, scales = int4.int4_quantize(np.asarray(W, np.float32).ravel())[:2]
            values = np.asarray(codes, np.float32) - np.float32(8)
        else:
            self.dev = q.quantize(to_dev(W), double_quant=kind == "dq")
            ow = OracleWeight(W, kind == "dq")
            values = np.asarray(nf4.NF4, np.float32)[ow.codes]
            scales = ow.scales
        a = np.repeat(np.asarray(scales, np.float32), 64)[: K * N]
        self.hat = S.f32_to_bf16_values(values * a).astype(np.float64).reshape(K, N)


class GatedCase:
    """Inputs of one gated block, on the host (fp64 of bf16 values) and the device."""

    def __init__(self, seed, M, K, N, r, kinds=("dq", "dq")):
        def normal(tid, shape, sigma):
            return S.normal(seed, M + 3 * K + 5 * N + 7 * r, tid, shape, sigma)
        self.M, self.K, self.N, self.r, self.c = M, K, N, r, 32.0 / max(r, 8)
        self.wg = DecodedWeight(normal(0, (K, N), 0.05), kinds[0])
        self.wu = DecodedWeight(normal(10, (K, N), 0.05), kinds[1])
        self.host = {"X": normal(1, (M, K), 1.0), "Ag": normal(2, (K, r), 0.05), "Bg": normal(3, (r, N), 0.05),
                     "Au": normal(12, (K, r), 0.05), "Bu": normal(13, (r, N), 0.05),
                     "dH": normal(4, (M, N), 1.0)}
        self.t = {n: to_dev(v) for n, v in self.host.items()}
        self.host = {n: np.asarray(v, np.float64) for n, v in self.host.items()}
        self.args = (self.wg.dev, self.wu.dev, self.t["Ag"], self.t["Bg"], self.t["Au"], self.t["Bu"], self.c)

    def branches(self):
        h = self.host
        return ((self.wg.hat, h["Ag"], h["Bg"]), (self.wu.hat, h["Au"], h["Bu"]))


def forward_bounds(case, kind):
    """(H, g, u, Zg, Zu), and how far the device's H, and its g and u before
    any rounding of their own, and its Z may be."""
    X, c, K, r = case.host["X"], case.c, case.K, case.r
    pre, pre_err, zs, z_err = [], [], [], []
    for W, A, B in case.branches():
        Z = c * (X @ A)
        dz = HALF * np.abs(Z) + abs(c) * gamma(K) * (np.abs(X) @ np.abs(A))
        pre.append(X @ W + Z @ B)
        pre_err.append(gamma(K + r) * (np.abs(X) @ np.abs(W) + np.abs(Z) @ np.abs(B)) + dz @ np.abs(B))
        zs.append(Z)
        z_err.append(SLACK * dz + TINY)
    g, u = pre
    dg, du = pre_err
    a, _ = act(g, kind)
    H = a * u
    # |act'| <= 1.13 for both functions
    err = 1.13 * dg * np.abs(u) + np.abs(a) * du + 1.13 * dg * du + FAST * np.abs(H) + HALF * np.abs(H)
    return (H, g, u, *zs), SLACK * err + TINY, [SLACK * e + TINY for e in pre_err], z_err


def backward_bounds(case, kind, X, g, u, Zg, Zu, grad_half):
    """The gradients from what the forward kept, and their bounds.  grad_half:
    the rounding of the adapters' gradients (0 for fp32)."""
    M, N, r, c, dH = case.M, case.N, case.r, case.c, case.host["dH"]
    a, d = act(g, kind)
    out, err = {"dX": 0.0}, {"dX": 0.0}
    for n, D, floor, (W, A, B), Z in zip(
            "gu", (dH * u * d, dH * a), (np.abs(dH * u), np.abs(dH * g)), case.branches(), (Zg, Zu)):
        # act and act' are off by FAST of 1 (of |g|) at most
        dD = HALF * np.abs(D) + FAST * 1.2 * floor
        dZ = c * (D @ B.T)
        ddZ = HALF * np.abs(dZ) + abs(c) * (dD @ np.abs(B).T + gamma(N) * (np.abs(D) @ np.abs(B).T))
        out["dX"] = out["dX"] + D @ W.T + dZ @ A.T
        err["dX"] = err["dX"] + dD @ np.abs(W).T + ddZ @ np.abs(A).T + gamma(2 * N + 2 * r) * (
            np.abs(D) @ np.abs(W).T + np.abs(dZ) @ np.abs(A).T)
        out["dA" + n] = X.T @ dZ
        err["dA" + n] = np.abs(X).T @ ddZ + gamma(M) * (np.abs(X).T @ np.abs(dZ))
        out["dB" + n] = Z.T @ D
        err["dB" + n] = np.abs(Z).T @ dD + gamma(M) * (np.abs(Z).T @ np.abs(D))
    for n in out:
        err[n] = SLACK * (err[n] + (HALF if n == "dX" else grad_half) * np.abs(out[n])) + TINY
    return out, err


def assert_within(name, got, ref, bound):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    over = np.abs(got - ref) - bound
    assert np.all(np.isfinite(got)), name
    if np.any(over > 0):
        at = np.unravel_index(np.argmax(over / bound), over.shape)
        raise AssertionError((name, at, got[at], ref[at], float(np.asarray(bound)[at])))
