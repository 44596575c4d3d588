"""The gated block on the GPU against the fp64 oracle, with element-wise bounds
that follow its roundings, and Frobenius bounds per matrix, row and tile."""
import numpy as np
import pytest
import torch

from oracle import act8 as oracle8
from tests._gpu_util import assert_close, to_np
from tests._operators_util import HALF, GatedCase, assert_within, backward_bounds, forward_bounds

pytestmark = pytest.mark.gpu


def _q():
    import bit_nf4_quantized_pack_b200 as q
    return q


FORWARD = [  # M, K, N, r, weights, act
    (1, 64, 64, 8, ("dq", "dq"), "silu"),
    (1, 1024, 704, 16, ("dq", "absmax"), "silu"),
    (4, 320, 192, 5, ("absmax", "absmax"), "gelu"),
    (16, 576, 1088, 64, ("dq", "dq"), "silu"),
    (17, 192, 64, 1, ("int4", "dq"), "gelu"),
    (64, 128, 320, 12, ("int4", "int4"), "silu"),
    (128, 256, 448, 33, ("dq", "dq"), "silu"),
    (129, 256, 128, 16, ("dq", "dq"), "gelu"),
    (257, 320, 192, 8, ("absmax", "dq"), "silu"),
    (300, 64, 320, 40, ("dq", "dq"), "silu"),
    (513, 192, 256, 16, ("dq", "dq"), "gelu"),
    (1100, 128, 64, 64, ("dq", "dq"), "silu"),
    # the rank-r products beside the fused GEMM
    (300, 1024, 320, 12, ("dq", "absmax"), "silu"),
    (600, 640, 192, 33, ("dq", "dq"), "gelu"),
    (1100, 1280, 128, 16, ("int4", "dq"), "silu"),
]


@pytest.mark.parametrize("M,K,N,r,kinds,act", FORWARD)
def test_forward(M, K, N, r, kinds, act):
    q = _q()
    case = GatedCase(11, M, K, N, r, kinds)
    (H, g, u, Zg, Zu), h_err, pre_err, z_err = forward_bounds(case, act)
    got, saved = q.gated_forward(case.t["X"], *case.args, act=act)
    assert saved is None
    assert_within("H", to_np(got), H, h_err)
    assert_close("H", to_np(got), H)
    kept, saved = q.gated_forward(case.t["X"], *case.args, act=act, save="bf16")
    assert torch.equal(got, kept)
    for n, t, ref, err in (("G", saved.G, g, pre_err[0]), ("U", saved.U, u, pre_err[1])):
        assert_within(n, to_np(t), ref, err + HALF * np.abs(ref) * 1.01)
    assert_within("Zg", to_np(saved.Zg), Zg, z_err[0])
    assert_within("Zu", to_np(saved.Zu), Zu, z_err[1])
    # the 8-bit form holds the checkpoints of exactly those bf16 matrices
    kept, saved8 = q.gated_forward(case.t["X"], *case.args, act=act, save="int8")
    assert torch.equal(got, kept)
    assert torch.equal(saved8.Zg, saved.Zg) and torch.equal(saved8.Zu, saved.Zu)
    for a, t in ((saved8.G, saved.G), (saved8.U, saved.U)):
        want = q.act8_quantize(t)
        assert torch.equal(a.codes, want.codes) and torch.equal(a.scales, want.scales)


BACKWARD = [  # M, K, N, r, weights, act, save, gradient type
    (1, 64, 64, 8, ("dq", "dq"), "silu", "bf16", torch.float32),
    (5, 320, 192, 5, ("absmax", "absmax"), "gelu", "int8", torch.bfloat16),
    (16, 576, 704, 64, ("dq", "absmax"), "silu", "bf16", torch.bfloat16),
    (65, 192, 64, 1, ("int4", "dq"), "gelu", "bf16", torch.float32),
    (129, 256, 448, 12, ("dq", "dq"), "silu", "int8", torch.float32),
    (257, 320, 192, 16, ("absmax", "dq"), "silu", "int8", torch.bfloat16),
    (300, 64, 320, 40, ("dq", "dq"), "gelu", "bf16", torch.bfloat16),
    (700, 576, 128, 64, ("dq", "dq"), "silu", "bf16", torch.float32),
    (1030, 448, 384, 12, ("dq", "dq"), "silu", "int8", torch.float32),
]


@pytest.mark.parametrize("M,K,N,r,kinds,act,save,dtype", BACKWARD)
def test_backward(M, K, N, r, kinds, act, save, dtype):
    q = _q()
    case = GatedCase(12, M, K, N, r, kinds)
    _, saved = q.gated_forward(case.t["X"], *case.args, act=act, save=save)
    X = q.act8_quantize(case.t["X"]) if save == "int8" else case.t["X"]
    got = q.gated_backward(case.t["dH"], X, saved, *case.args, act=act, grad_dtype=dtype)

    def host(t):
        if isinstance(t, q.Act8):
            return oracle8.act8_dequantize(t.codes.cpu().numpy(), t.scales.cpu().numpy())
        return to_np(t)
    ref, err = backward_bounds(case, act, host(X), host(saved.G), host(saved.U), host(saved.Zg), host(saved.Zu),
                               HALF if dtype == torch.bfloat16 else 0.0)
    for n, t in zip(("dX", "dAg", "dBg", "dAu", "dBu"), got):
        assert t.dtype == (torch.bfloat16 if n == "dX" else dtype)
        assert_within(n, to_np(t), ref[n], err[n])
        assert_close(n, to_np(t), ref[n])


def test_gradients_are_the_differences():
    """dX against differences of the operator itself: H's bf16 rounding limits
    the step, so the direction is the gradient's own and the step large enough
    for it to show; the second-order term is measured by halving the step."""
    q = _q()
    case = GatedCase(13, 40, 128, 192, 8)
    H, saved = q.gated_forward(case.t["X"], *case.args, save="bf16")
    dX = q.gated_backward(case.t["dH"], case.t["X"], saved, *case.args)[0]
    v = torch.sign(dX.float())
    base, dH = case.t["X"].float(), case.t["dH"].double()
    slopes = []
    for h in (2.0 ** -4, 2.0 ** -5):
        hi, lo = (base + h * v).to(torch.bfloat16), (base - h * v).to(torch.bfloat16)
        # what the rounding of the inputs made of the step
        step = (hi.double() - lo.double())
        diff = ((q.gated_forward(hi, *case.args)[0].double() - q.gated_forward(lo, *case.args)[0].double()) * dH).sum()
        slopes.append(((diff - (dX.double() * step).sum()) / (dX.double() * step).sum().abs()).item())
    # H's rounding is random: half a step (2^-8) of |H dH| over 40 * 192 values,
    # root sum of squares, against the change itself, and the curvature is
    # cubic in h (central differences)
    noise = (2.0 ** -8 * (H.double() * dH).square().sum().sqrt() * 2 / (dX.double().abs().sum() * 2 * 2.0 ** -5)).item()
    curve = abs(slopes[0] - slopes[1]) * 4 / 3
    assert abs(slopes[1]) <= 4 * noise + curve + 2.0 ** -8


@pytest.mark.parametrize("M", [1, 130])
def test_extremes(M):
    """Saturated and vanishing gates, zero adapters, a zero token."""
    q = _q()
    case = GatedCase(14, M, 64, 128, 8)
    X = case.t["X"] * 256                      # exact in bf16
    X[0] = 0
    zero = torch.zeros_like(case.t["Bg"])
    case.host.update(X=to_np(X), Bg=np.zeros_like(case.host["Bg"]), Bu=np.zeros_like(case.host["Bu"]))
    for act in ("silu", "gelu"):
        H, saved = q.gated_forward(X, *case.args[:3], zero, case.args[4], zero, case.c, act=act, save="bf16")
        assert torch.isfinite(H).all() and not H[0].any()
        ref, err, _, _ = forward_bounds(case, act)
        assert_within("H", to_np(H), ref[0], err)
        grads = q.gated_backward(case.t["dH"], X, saved, *case.args[:3], zero, case.args[4], zero, case.c, act=act)
        assert all(torch.isfinite(t).all() for t in grads)
        assert not grads[1].any() and not grads[3].any()      # dZ = 0 with B = 0


def test_nonfinite_input_reaches_only_its_row():
    q = _q()
    for M in (3, 200):
        case = GatedCase(15, M, 128, 64, 8)
        want, _ = q.gated_forward(case.t["X"], *case.args)
        X = case.t["X"].clone()
        X[1, 5] = float("nan")
        H, _ = q.gated_forward(X, *case.args)
        assert torch.isnan(H[1]).all()
        rows = [i for i in range(M) if i != 1]
        assert torch.equal(H[rows], want[rows])


def test_outputs_stay_inside_and_repeat():
    q = _q()
    for M, N in ((1, 64), (77, 192), (300, 320)):
        case = GatedCase(16, M, 192, N, 12)
        pad = 4096

        def guarded(shape, dtype=torch.bfloat16):
            n = int(np.prod(shape))
            big = torch.full((n + 2 * pad,), 5, dtype=dtype, device="cuda")
            return big, big[pad:pad + n].view(shape)
        bufs = [guarded((M, N))]
        saved = []
        for _ in range(2):
            bufs += [guarded((M, N), torch.int8), guarded((M, N // 64), torch.float32)]
            saved.append(q.Act8(bufs[-2][1], bufs[-1][1]))
        bufs += [guarded((M, 12)), guarded((M, 12))]
        kept = q.GatedSaved(saved[0], saved[1], bufs[-2][1], bufs[-1][1])
        H, _ = q.gated_forward(case.t["X"], *case.args, H=bufs[0][1], saved=kept)
        grads = [guarded((M, 192)), guarded((192, 12)), guarded((12, N)), guarded((192, 12)), guarded((12, N))]
        out = dict(zip(("dX", "dAg", "dBg", "dAu", "dBu"), (g[1] for g in grads)))
        q.gated_backward(case.t["dH"], case.t["X"], kept, *case.args, grad_dtype=torch.bfloat16, **out)
        torch.cuda.synchronize()
        for big, t in bufs + grads:
            assert (big[:pad] == 5).all() and (big[pad + t.numel():] == 5).all()
        # the same bits again
        H2, kept2 = q.gated_forward(case.t["X"], *case.args, save="int8")
        again = q.gated_backward(case.t["dH"], case.t["X"], kept2, *case.args, grad_dtype=torch.bfloat16)
        assert torch.equal(H, H2) and all(torch.equal(a, b) for a, b in zip(again, out.values()))


@pytest.mark.parametrize("M,K,N,r,dq", [(1, 4096, 11008, 16, True), (16, 2048, 22016, 64, False),
                                        (128, 4096, 4160, 8, True), (70, 1088, 11008, 24, True),
                                        (200, 4096, 11008, 16, True)])
def test_forward_at_full_width(M, K, N, r, dq):
    """Long runs of units per SM, against fp64 products of the dequantized
    weights on the device: the bound of the small cases, the decode's own
    double rounding (one bf16 step of one weight in 2^16) aside, which Frobenius
    norms do not see."""
    q = _q()
    g = torch.Generator(device="cuda").manual_seed(M + N)

    def t(*shape, sigma):
        return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)
    X, c = t(M, K, sigma=1.0), 2.0
    W = [q.quantize(t(K, N, sigma=0.02), double_quant=dq) for _ in range(2)]
    A, B = [t(K, r, sigma=0.02) for _ in range(2)], [t(r, N, sigma=0.02) for _ in range(2)]
    pre = []
    for i in range(2):
        Z = (c * (X.double() @ A[i].double()))
        pre.append(X.double() @ q.dequantize(W[i]).double() + Z @ B[i].double())
    want = pre[0] * torch.sigmoid(pre[0]) * pre[1]
    for _ in range(3):
        H, saved = q.gated_forward(X, W[0], W[1], A[0], B[0], A[1], B[1], c, save="bf16")
        for got, ref in ((H, want), (saved.G, pre[0]), (saved.U, pre[1])):
            rel = ((got.double() - ref).norm() / ref.norm()).item()
            # one rounding to bf16: 2^-8 / sqrt(3) at most in this norm, and Z's
            # on the small adapter term
            assert rel <= 2.0 ** -8, rel
            assert ((got.double() - ref).abs().max() / ref.abs().max()).item() <= 2.0 ** -7
