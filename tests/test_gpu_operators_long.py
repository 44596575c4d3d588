"""Matrices of more than 2^31 elements: rows whose offsets need 64 bits, against
fp64 on sampled rows (among them the two around element 2^31) and, for the
adapters' gradients, over all rows.  Bounds as derived for a full step: a
rounding to bf16 is 2^-8 / sqrt(3) of the value at most in the root mean square,
three in a row 3.9e-3 of a Frobenius norm.  About 25 GB."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TOL = 5e-3
M, WIDE, R = 200003, 11008, 8
AROUND = 2 ** 31 // WIDE
ROWS = [0, 1, 99999, AROUND - 1, AROUND, AROUND + 1, M - 2, M - 1]
STEP = 20000


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def _q():
    import bit_nf4_quantized_pack_b200 as q
    return q


def bf16(*shape, sigma=1.0):
    return torch.randn(*shape, device="cuda", dtype=torch.bfloat16) * sigma


def rel(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


def over_rows(a, b):
    """aᵀ·b in fp64, in pieces of the rows."""
    return sum(a[i:i + STEP].double().T @ b[i:i + STEP].double() for i in range(0, M, STEP))


def test_wide_outputs():
    q = _q()
    K = 64
    torch.manual_seed(1)
    rows = torch.tensor(ROWS, device="cuda")
    w = [q.quantize(bf16(K, WIDE, sigma=0.05)) for _ in range(2)]
    A, B = [bf16(K, R, sigma=0.05) for _ in range(2)], [bf16(R, WIDE, sigma=0.05) for _ in range(2)]
    W = [q.dequantize(x).double() for x in w]
    X, args = bf16(M, K), (w[0], w[1], A[0], B[0], A[1], B[1], 1.0)
    H, saved = q.gated_forward(X, *args, save="int8")

    def at(a):
        return q.act8_dequantize(q.Act8(a.codes[rows].contiguous(), a.scales[rows].contiguous())).double()
    x = X[rows].double()
    pre = [x @ W[i] + (x @ A[i].double()) @ B[i].double() for i in range(2)]
    assert rel(H[rows], torch.nn.functional.silu(pre[0]) * pre[1]) <= TOL
    for a, p in zip((saved.G, saved.U), pre):
        # half a code of 127 of the block's largest value at most, and two roundings
        top = p.abs().view(len(ROWS), -1, 64).amax(2, keepdim=True).expand(-1, -1, 64).reshape(p.shape)
        assert ((at(a) - p).abs() <= top * (0.5 / 127 * 1.01 + 2.0 ** -8 * 2) + 1e-6).all()
    a8 = q.act8_quantize(H)
    few = q.act8_quantize(H[rows].contiguous())
    assert torch.equal(a8.codes[rows], few.codes) and torch.equal(a8.scales[rows], few.scales)
    assert torch.equal(q.act8_dequantize(a8)[rows], q.act8_dequantize(few))
    del a8, H
    dH = bf16(M, WIDE)
    dX = q.gated_backward(dH, X, saved, *args)[0]
    G, U, d = at(saved.G), at(saved.U), dH[rows].double()
    s = torch.sigmoid(G)
    D = [d * U * (s + G * s * (1 - s)), d * G * s]
    want = sum(D[i] @ W[i].T + (D[i] @ B[i].double().T) @ A[i].double().T for i in range(2))
    assert rel(dX[rows], want) <= TOL
    dX, _, dB = q.linear_backward(dH, q.act8_quantize(X), saved.Zg, w[0], A[0], B[0], 1.0)
    assert rel(dX[rows], d @ W[0].T + (d @ B[0].double().T) @ A[0].double().T) <= TOL
    assert rel(dB, over_rows(saved.Zg, dH)) <= TOL


def test_wide_inputs():
    q = _q()
    N = 64
    torch.manual_seed(2)
    rows = torch.tensor(ROWS, device="cuda")
    w, A, B = q.quantize(bf16(WIDE, N, sigma=0.02)), bf16(WIDE, R, sigma=0.02), bf16(R, N, sigma=0.05)
    W = q.dequantize(w).double()
    X, dY, Zc = bf16(M, WIDE), bf16(M, N), bf16(M, R)
    a8 = q.act8_quantize(X)
    dZ = dY.double() @ B.double().T
    for x, value in ((X, X), (a8, q.act8_dequantize(a8))):
        dX, dA, _ = q.linear_backward(dY, x, Zc, w, A, B, 1.0, grad_dtype=torch.bfloat16)
        assert rel(dX[rows], dY[rows].double() @ W.T + dZ[rows] @ A.double().T) <= TOL
        assert rel(dA, over_rows(value, dZ)) <= TOL
    y = torch.randint(N, (M,), device="cuda")
    loss, lse = q.head_loss_forward(X, w, y)
    x = X[rows].double()
    logits = x @ W
    ref = torch.logsumexp(logits, 1)
    bound = WIDE * 2.0 ** -23 * (x.abs() @ W.abs()).amax(1) + 2.0 ** -18 * (1 + ref.abs())
    assert ((lse[rows].double() - ref).abs() <= bound).all()
    dX = q.head_loss_backward(torch.ones(M, device="cuda"), X, lse, w, y)
    p = torch.softmax(logits, 1)
    p[torch.arange(len(ROWS), device="cuda"), y[rows]] -= 1
    assert rel(dX[rows], p @ W.T) <= 2.0 ** -8 + 2.0 ** -8 / 3 ** 0.5
