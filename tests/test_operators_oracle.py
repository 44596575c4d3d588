"""Pins of the oracles of the gated block, the 8-bit checkpoints and the head
loss: central differences, hand-written cases and error bounds."""
import numpy as np
import pytest

from inputs import synthetic as S
from oracle import act8, gated, loss


def _rng(*key):
    return np.random.default_rng(list(key))


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_gradients_are_the_differences(kind):
    g = _rng(1, len(kind))
    M, K, N, r, c = 3, 4, 5, 2, 0.7
    t = {n: g.normal(size=s) for n, s in dict(X=(M, K), Wg=(K, N), Wu=(K, N), Ag=(K, r), Bg=(r, N),
                                              Au=(K, r), Bu=(r, N)).items()}
    dH = g.normal(size=(M, N))
    order = ("X", "Wg", "Wu", "Ag", "Bg", "Au", "Bu")

    def value(t):
        return float((gated.gated_forward(*(t[n] for n in order), c, kind)[0] * dH).sum())

    _, gp, u, Zg, Zu = gated.gated_forward(*(t[n] for n in order), c, kind)
    grads = dict(zip(("X", "Ag", "Bg", "Au", "Bu"),
                     gated.gated_backward(dH, t["X"], gp, u, *(t[n] for n in order[1:]), c, kind)))
    assert np.allclose(Zg, c * t["X"] @ t["Ag"]) and np.allclose(Zu, c * t["X"] @ t["Au"])
    h = 1e-5
    for n, grad in grads.items():
        for idx in np.ndindex(*t[n].shape):
            lo, hi = {**t, n: t[n].copy()}, {**t, n: t[n].copy()}
            lo[n][idx] -= h
            hi[n][idx] += h
            # central differences: error of order h^2 and 1e-16 / h
            assert abs((value(hi) - value(lo)) / (2 * h) - grad[idx]) < 1e-7 * (1 + abs(grad[idx])), n


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_values(kind):
    a, d = gated.act(np.array([0.0, 50.0, -50.0]), kind)
    assert a[0] == 0 and d[0] == 0.5
    assert abs(a[1] - 50) < 1e-12 and abs(d[1] - 1) < 1e-12
    assert abs(a[2]) < 1e-18 and abs(d[2]) < 1e-18


def test_loss_gradient_is_the_difference():
    g = _rng(2)
    M, K, V = 4, 3, 7
    X, W = g.normal(size=(M, K)), g.normal(size=(K, V + 2))
    labels = np.array([0, 6, -100, 3])
    dl = g.normal(size=M)
    dX = loss.head_loss_backward(dl, X, W, labels, V)
    h = 1e-5
    for idx in np.ndindex(M, K):
        lo, hi = X.copy(), X.copy()
        lo[idx] -= h
        hi[idx] += h
        num = ((loss.head_loss_forward(hi, W, labels, V)[0] - loss.head_loss_forward(lo, W, labels, V)[0]) * dl).sum() / (2 * h)
        assert abs(num - dX[idx]) < 1e-7
    assert not dX[2].any()


def test_loss_of_uniform_logits():
    lo, lse = loss.head_loss_forward(np.zeros((2, 4)), np.ones((4, 64)), np.array([0, 9]), 10)
    assert np.allclose(lse, np.log(10)) and np.allclose(lo, np.log(10))


def test_act8_codes_and_values():
    x = np.zeros((2, 128), np.float32)
    x[0, :64] = np.linspace(-1, 1, 64)
    x[0, 64] = 254.0          # scale 2: 3 and 5 sit on ties, to the even code
    x[0, 65], x[0, 66], x[0, 67] = 3.0, 5.0, -3.0
    x[1, 64:] = 2.0 ** -133   # amax / 127 below the normal range: scale 1
    x = S.f32_to_bf16_values(x)
    codes, s = act8.act8_quantize(x)
    assert s[0, 1] == 2 and list(codes[0, 64:68]) == [127, 2, 2, -2]
    assert s[1, 0] == 1 and s[1, 1] == 1 and not codes[1].any()
    assert codes[0, 0] == -127 and codes[0, 63] == 127
    v = act8.act8_dequantize(codes, s)
    # half a code step, and the bf16 rounding of the value (half a step: 2^-8)
    assert np.all(np.abs(v[0] - x[0]) <= np.repeat(s[0], 64) / 2 * (1 + 2 ** -20) + np.abs(v[0]) * 2 ** -8)


def test_act8_is_stable():
    """Quantizing the values again gives the same codes where the scale is a
    power of two (each value is then an exact bf16)."""
    g = _rng(3)
    x = S.f32_to_bf16_values((g.integers(-127, 128, (4, 192)) * 0.25).astype(np.float32))
    x[:, ::64] = 31.75
    codes, s = act8.act8_quantize(x)
    assert np.all(s == 0.25) and np.array_equal(act8.act8_dequantize(codes, s), x)
