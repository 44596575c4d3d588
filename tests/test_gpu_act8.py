"""8-bit activation checkpoints on the GPU: the codec bit for bit, and the
backward of a layer from its input's codes."""
import numpy as np
import pytest
import torch

from inputs import synthetic as S
from oracle import act8 as oracle
from tests._gpu_util import assert_close, to_dev, to_np
from tests._operators_util import HALF, SLACK, TINY, DecodedWeight, assert_within, gamma

pytestmark = pytest.mark.gpu


def _q():
    import bit_nf4_quantized_pack_b200 as q
    return q


def _matrix(M, K, seed=5):
    g = np.random.default_rng([seed, M, K])
    x = g.normal(size=(M, K)) * np.exp(g.normal(size=(M, 1)) * 3)
    x[g.random((M, K)) < 0.01] *= 50
    x[:, : 64][g.random((M, 1))[:, 0] < 0.3] = 0            # all-zero blocks
    return S.f32_to_bf16_values(x.astype(np.float32))


@pytest.mark.parametrize("M,K", [(1, 64), (3, 192), (37, 64), (5, 4096), (129, 320), (1000, 11008)])
def test_codec_is_bit_exact(M, K):
    q = _q()
    x = _matrix(M, K)
    X = to_dev(x)
    a = q.act8_quantize(X)
    codes, scales = oracle.act8_quantize(x)
    assert np.array_equal(a.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(a.codes.cpu().numpy(), codes)
    assert np.array_equal(to_np(q.act8_dequantize(a)), oracle.act8_dequantize(codes, scales))


def test_codec_ties_and_extremes():
    q = _q()
    x = np.zeros((4, 128), np.float32)
    x[0, 0], x[0, 1:6] = 254.0, (3.0, 5.0, -3.0, -5.0, 251.0)           # scale 2: exact ties
    x[0, 64:] = np.finfo(np.float32).tiny / 128                          # below the normal range
    x[1, :64] = 3.3895313892515355e38                                    # the largest bf16
    x[1, 64:] = np.arange(64) * 2.0 ** -120                              # a small scale
    x[2, 70] = -1.0
    x[3] = np.random.default_rng(8).integers(-127, 128, 128) + 0.5       # many values near ties
    x = S.f32_to_bf16_values(x)
    a = q.act8_quantize(to_dev(x))
    codes, scales = oracle.act8_quantize(x)
    assert np.array_equal(a.codes.cpu().numpy(), codes)
    assert np.array_equal(a.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(to_np(q.act8_dequantize(a)), oracle.act8_dequantize(codes, scales))


def test_codec_over_all_significands_and_magnitudes():
    """Every pair of significands of a value and its block's largest magnitude, the
    values up to eight binades below; and blocks through all binades of bf16."""
    q = _q()
    sig = np.arange(128, 256) / 128.0
    values = np.concatenate([sig * 2.0 ** -e for e in range(9)])
    values = np.resize(np.concatenate([values, -values]), 63 * 37)
    rows = []
    for top in sig:
        block = np.empty((37, 64))
        block[:, 0] = top
        block[:, 1:] = values.reshape(37, 63)
        rows.append(np.where(np.abs(block) <= top, block, 0).reshape(-1))
    g = np.random.default_rng(3)
    for e in range(-133, 127, 2):
        block = g.choice(sig, (37, 64)) * 2.0 ** (e - g.integers(0, 9, (37, 64))) * g.choice([-1, 1], (37, 64))
        rows.append(block.reshape(-1))
    x = S.f32_to_bf16_values(np.array(rows).astype(np.float32))
    a = q.act8_quantize(to_dev(x))
    codes, scales = oracle.act8_quantize(x)
    assert np.array_equal(a.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(a.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_codec_reports_nonfinite(bad):
    q = _q()
    X = torch.randn(9, 256, device="cuda").to(torch.bfloat16)
    X[8, 200] = bad
    st = q.new_status()
    q.act8_quantize(X, status=st)
    assert q.status_sync(st)[0] == 3
    with pytest.raises(q.QLoRAError):
        q.act8_quantize(X)


def test_codec_writes_only_its_rows():
    q = _q()
    big = q.Act8(torch.full((7, 192), 77, dtype=torch.int8, device="cuda"),
                 torch.full((16, 3), -3.0, device="cuda"))
    x = _matrix(2, 192)
    # rows 2 and 3 of the codes; scales from element 12 (a 16-byte boundary) on
    out = q.Act8(big.codes[2:4], big.scales[4:6])
    q.act8_quantize(to_dev(x), out=out)
    codes, scales = oracle.act8_quantize(x)
    assert np.array_equal(out.codes.cpu().numpy(), codes) and np.array_equal(out.scales.cpu().numpy(), scales)
    assert (big.codes[:2] == 77).all() and (big.codes[4:] == 77).all()
    assert (big.scales[:4] == -3).all() and (big.scales[6:] == -3).all()


CASES = [  # M, K, N, r, weight, gradient type
    (1, 64, 64, 8, "dq", torch.float32),
    (37, 192, 128, 5, "absmax", torch.bfloat16),
    (129, 320, 192, 16, "dq", torch.bfloat16),
    (300, 256, 704, 64, "int4", torch.float32),
    (1000, 448, 64, 1, "dq", torch.bfloat16),
]


@pytest.mark.parametrize("M,K,N,r,kind,dtype", CASES)
def test_layer_backward_from_codes(M, K, N, r, kind, dtype):
    q = _q()
    lin = S.random_case(M + K + N + r, M, K, N, r)
    dY = np.asarray(S.normal(7, M, 4, (M, N), 1.0))
    Zc = np.asarray(S.normal(8, M, 6, (M, r), 1.0))
    w = DecodedWeight(lin.W, kind)
    c = 0.75
    a = q.act8_quantize(to_dev(lin.X))
    args = (to_dev(dY), a, to_dev(Zc), w.dev, to_dev(lin.A), to_dev(lin.B), c)
    dX, dA, dB = q.linear_backward(*args, grad_dtype=dtype)
    assert dA.dtype == dB.dtype == dtype
    X = oracle.act8_dequantize(*oracle.act8_quantize(lin.X))
    dY, Zc, A, B = (np.asarray(v, np.float64) for v in (dY, Zc, lin.A, lin.B))
    half = HALF if dtype == torch.bfloat16 else 0.0
    dZ = c * dY @ B.T
    ddZ = HALF * np.abs(dZ) + c * gamma(N) * (np.abs(dY) @ np.abs(B).T)
    ref = {"dX": dY @ w.hat.T + dZ @ A.T, "dA": X.T @ dZ, "dB": Zc.T @ dY}
    err = {"dX": gamma(N + r) * (np.abs(dY) @ np.abs(w.hat).T + np.abs(dZ) @ np.abs(A).T) + ddZ @ np.abs(A).T
           + HALF * np.abs(ref["dX"]),
           "dA": np.abs(X).T @ ddZ + gamma(M) * np.abs(X).T @ np.abs(dZ) + half * np.abs(ref["dA"]),
           "dB": gamma(M) * np.abs(Zc).T @ np.abs(dY) + half * np.abs(ref["dB"])}
    for n, got in (("dX", dX), ("dA", dA), ("dB", dB)):
        assert_within(n, to_np(got), ref[n], SLACK * err[n] + TINY)
        assert_close(n, to_np(got), ref[n])
    # the same gradients as from the bf16 matrix that the codes stand for; dA may
    # come from a kernel that adds in another order: each of the two is the
    # rounding (HALF) of a sum of the same products within gamma(M) of the exact
    dX8, dA8, dB8 = q.linear_backward(*args, grad_dtype=torch.bfloat16)
    dXf, dAf, dBf = q.linear_backward(args[0], q.act8_dequantize(a), *args[2:], grad_dtype=torch.bfloat16)
    assert torch.equal(dX8, dXf) and torch.equal(dB8, dBf)
    sums = gamma(M) * np.abs(X).T @ (np.abs(dZ) + ddZ)
    assert_within("dA of both", to_np(dA8), to_np(dAf), 2 * SLACK * (sums + HALF * (np.abs(to_np(dAf)) + sums)) + TINY)


def test_gradients_in_bf16_are_the_rounded_fp32_ones():
    """Both types come from the same fp32 sums where the same kernels form them."""
    q = _q()
    M, K, N, r = 300, 256, 320, 16
    lin = S.random_case(9, M, K, N, r)
    w = DecodedWeight(lin.W, "dq")
    a = q.act8_quantize(to_dev(lin.X))
    dY, Zc = to_dev(S.normal(7, M, 4, (M, N), 1.0)), to_dev(S.normal(8, M, 6, (M, r), 1.0))
    args = (dY, a, Zc, w.dev, to_dev(lin.A), to_dev(lin.B), 2.0)
    wide = q.linear_backward(*args)
    narrow = q.linear_backward(*args, grad_dtype=torch.bfloat16)
    assert torch.equal(wide[0], narrow[0])
    for x, y in zip(wide[1:], narrow[1:]):
        assert torch.equal(x.to(torch.bfloat16), y)
