"""The operators at sizes where the fused GEMM and its neighbours work as they
do in a full training step: tiles of 512 rows with both accumulators, several
tiles per CTA pair, contractions cut into items that do not divide evenly,
rank-r products with several row tiles per CTA, gradients on the library's own
stream, several pieces of the vocabulary.

References are fp64 products on the device of what the calls received.  A
rounding to bf16 is off by at most 2^-8 of the value and, over many values, by
2^-8 / sqrt(3) in the root mean square at most (uniform within half a step, the
value at the bottom of its binade).  Two such roundings in a row (an operand's,
the result's) give 3.2e-3 of the Frobenius norm, three 3.9e-3; 5e-3 leaves room
for the smaller terms (sums in fp32, 2^-18 of the activation's exponential, the
adapters' share) and for the blocks of 128 x 256 over which it is also asked.
A K-step left out or counted twice is far above it: one of n changes a sum of
random products by about n^-1/2, 3e-2 for the longest contraction here.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TOL = 5e-3


def _q():
    import bit_nf4_quantized_pack_b200 as q
    return q


def bf16(g, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)


def close(name, got, ref, tol=TOL):
    """Frobenius norms of the whole and of every block of 128 rows x 256 columns."""
    got = got.double()
    assert got.shape == ref.shape and torch.isfinite(got).all(), name
    d, r = (got - ref).square(), ref.square()
    rel = (d.sum() / r.sum()).sqrt().item()
    assert rel <= tol, (name, rel)
    rows, cols = -(-ref.shape[0] // 128) * 128, -(-ref.shape[1] // 256) * 256
    pad = (0, cols - ref.shape[1], 0, rows - ref.shape[0])
    d, r = (torch.nn.functional.pad(t, pad).view(rows // 128, 128, cols // 256, 256).sum((1, 3)) for t in (d, r))
    # a block's own figure where it has its share of the values (a ragged edge may
    # hold a few only, whose root mean square is not settled)
    full = torch.nn.functional.pad(torch.ones_like(ref), pad).view(rows // 128, 128, cols // 256, 256).sum((1, 3))
    worst = torch.where(full >= 256, (d / r.clamp(min=1e-300)).sqrt(), torch.zeros_like(d)).max().item()
    assert worst <= 1.2 * tol, (name, worst)


def act64(g, kind):
    """act(g) and its derivative."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    k = np.sqrt(2 / np.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


GATED = [  # M, K, N, r, act, save, gradient type
    # forward tiles of 512 rows (the last with six); a split dX in four even items
    (1030, 1088, 11008, 24, "silu", "int8", torch.bfloat16),
    # in items of 87 K-steps of 346, the second in both weights, the last of 85
    (1030, 1088, 11072, 5, "gelu", "bf16", torch.float32),
    # forward's rank-r products with two row tiles a CTA; a split dX in two items, one a weight
    (1000, 4096, 8960, 16, "silu", "bf16", torch.float32),
    # dX: two tiles a pair, the last of 216 rows; dZ with three row tiles a CTA
    (3800, 4096, 4096, 64, "silu", "int8", torch.float32),
    # items of 9 K-steps of 86, the fifth in both weights, the last of 5
    (333, 1088, 2752, 12, "gelu", "int8", torch.bfloat16),
]


@pytest.mark.parametrize("M,K,N,r,act,save,dtype", GATED)
def test_gated_step(M, K, N, r, act, save, dtype):
    q = _q()
    g = torch.Generator(device="cuda").manual_seed(M + N + r)
    X, dH, c = bf16(g, M, K), bf16(g, M, N), 2.0
    w = [q.quantize(bf16(g, K, N, sigma=0.02)) for _ in range(2)]
    A, B = [bf16(g, K, r, sigma=0.02) for _ in range(2)], [bf16(g, r, N, sigma=0.05) for _ in range(2)]
    args = (w[0], w[1], A[0], B[0], A[1], B[1], c)
    W = [q.dequantize(x).double() for x in w]
    H, saved = q.gated_forward(X, *args, act=act, save="bf16")
    pre = [X.double() @ W[i] + (c * (X.double() @ A[i].double())) @ B[i].double() for i in range(2)]
    for name, got, ref in (("G", saved.G, pre[0]), ("U", saved.U, pre[1]), ("H", H, act64(pre[0], act)[0] * pre[1])):
        close(name, got, ref)
    if save == "int8":
        H8, saved8 = q.gated_forward(X, *args, act=act, save="int8")
        assert torch.equal(H, H8) and torch.equal(saved.Zg, saved8.Zg) and torch.equal(saved.Zu, saved8.Zu)
        for a, t in ((saved8.G, saved.G), (saved8.U, saved.U)):
            want = q.act8_quantize(t)
            assert torch.equal(a.codes, want.codes) and torch.equal(a.scales, want.scales)
        saved = saved8
    x = q.act8_quantize(X) if save == "int8" else X
    value = lambda t: (q.act8_dequantize(t) if isinstance(t, q.Act8) else t).double()   # noqa: E731
    G, U, Xv = value(saved.G), value(saved.U), value(x)
    a, d = act64(G, act)
    D = [dH.double() * U * d, dH.double() * a]
    dZ = [c * (D[i] @ B[i].double().T) for i in range(2)]
    Z = [saved.Zg.double(), saved.Zu.double()]
    ref = [sum(D[i] @ W[i].T + dZ[i] @ A[i].double().T for i in range(2)),
           Xv.T @ dZ[0], Z[0].T @ D[0], Xv.T @ dZ[1], Z[1].T @ D[1]]
    first = None
    for _ in range(2):
        grads = q.gated_backward(dH, x, saved, *args, act=act, grad_dtype=dtype)
        for name, got, want in zip(("dX", "dAg", "dBg", "dAu", "dBu"), grads, ref):
            close(name, got, want)
        if first is not None:
            assert all(torch.equal(s, t) for s, t in zip(first, grads))
        first = grads


LOSS = [  # M, K, vocab
    (200, 256, 1200),      # dX in two items of 10 of 19 steps
    (300, 256, 2230),      # four items of 9 of 35
    (3800, 4096, 1000),    # dX: two tiles a pair
    (3800, 4096, 20001),   # the same in two pieces, whose sums meet in fp32
    (1030, 512, 70001),    # two pieces and few tiles
]


@pytest.mark.parametrize("M,K,vocab", LOSS)
def test_loss_and_gradient(M, K, vocab):
    q = _q()
    g = torch.Generator(device="cuda").manual_seed(M + vocab)
    N = -(-vocab // 64) * 64
    # logits of a few units, so that the softmax has some heavy tokens in every row
    X, w = bf16(g, M, K, sigma=4 / (0.02 * K ** 0.5)), q.quantize(bf16(g, K, N, sigma=0.02))
    labels = torch.randint(vocab, (M,), generator=g, device="cuda")
    labels[::9] = -100
    labels[1] = vocab - 1
    dloss = torch.randn(M, generator=g, device="cuda")
    W = q.dequantize(w).double()[:, :vocab]
    logits = X.double() @ W
    lse_ref = torch.logsumexp(logits, 1)
    at = labels.clamp(min=0)[:, None]
    counted = labels >= 0
    loss_ref = (lse_ref - logits.gather(1, at)[:, 0]) * counted
    # a logit is off by at most K 2^-23 of the sum of its products' magnitudes
    dl = K * 2.0 ** -23 * (X.double().abs() @ W.abs()).amax(1)
    p = torch.exp(logits - lse_ref[:, None])
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=p.dtype))
    dX_ref = (p * (dloss.double() * counted)[:, None]) @ W.T
    del logits, p
    first = None
    for _ in range(2):
        loss, lse = q.head_loss_forward(X, w, labels, vocab=vocab)
        assert ((lse.double() - lse_ref).abs() <= dl + 2.0 ** -18 * (1 + lse_ref.abs())).all()
        assert ((loss.double() - loss_ref).abs() <= 2 * dl + 2.0 ** -18 * (1 + loss_ref.abs())).all()
        dX = q.head_loss_backward(dloss, X, lse, w, labels, vocab=vocab)
        # the label's element of P is near -1 in most rows, where bf16's half step is
        # 2^-9 to 2^-8 of it, and alike in all of them: 2^-8, and the result's rounding
        close("dX", dX, dX_ref, tol=2.0 ** -8 + 2.0 ** -8 / 3 ** 0.5)
        assert not dX[labels < 0].any()
        if first is not None:
            assert all(torch.equal(s, t) for s, t in zip(first, (loss, lse, dX)))
        first = (loss, lse, dX)


@pytest.mark.parametrize("M,K,N,r,is8,dtype", [(1500, 4096, 4096, 16, True, torch.bfloat16),
                                               (1500, 4096, 4096, 16, False, torch.bfloat16),
                                               (1111, 11008, 1088, 5, True, torch.float32)])
def test_linear_backward_on_the_side_stream(M, K, N, r, is8, dtype):
    q = _q()
    assert M * K * N >= 1e10
    g = torch.Generator(device="cuda").manual_seed(M + K)
    X, dY, Zc, c = bf16(g, M, K), bf16(g, M, N), bf16(g, M, r), 0.5
    w, A, B = q.quantize(bf16(g, K, N, sigma=0.02)), bf16(g, K, r, sigma=0.02), bf16(g, r, N, sigma=0.02)
    x = q.act8_quantize(X) if is8 else X
    Xv = (q.act8_dequantize(x) if is8 else X).double()
    dZ = c * (dY.double() @ B.double().T)
    ref = (dY.double() @ q.dequantize(w).double().T + dZ @ A.double().T, Xv.T @ dZ, Zc.double().T @ dY.double())
    first = None
    for _ in range(2):
        grads = q.linear_backward(dY, x, Zc, w, A, B, c, grad_dtype=dtype)
        for name, got, want in zip(("dX", "dA", "dB"), grads, ref):
            assert got.dtype == (torch.bfloat16 if name == "dX" else dtype)
            close(name, got, want)
        if first is not None:
            assert all(torch.equal(s, t) for s, t in zip(first, grads))
        first = grads
