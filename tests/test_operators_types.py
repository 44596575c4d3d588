"""Arguments of the operators that are no tensor, no weight or no saved state at
all: TypeError, as for a tensor of a wrong type."""
import pytest
import torch


@pytest.fixture(scope="module")
def q():
    from tests.conftest import ensure_built
    ensure_built()
    import bit_nf4_quantized_pack_b200
    return bit_nf4_quantized_pack_b200


def test_checks(q):
    from bit_nf4_quantized_pack_b200 import _args, act8, gated
    cpu, t = torch.device("cpu"), torch.zeros(64, 128, dtype=torch.bfloat16)
    for call in (lambda: _args.weight(None, "w", 64, 128, cpu), lambda: _args.weight(t, "w", 64, 128, cpu),
                 lambda: _args.columns((64, 128), "w"), lambda: act8.width(None, "X"),
                 lambda: act8.width(q.Act8(None, None), "X"), lambda: gated._kept((t, t, t, t), 64, 128, 8, cpu),
                 lambda: gated._kept(None, 64, 128, 8, cpu), lambda: gated._weights(64, cpu, None, None, t, t, t, t),
                 lambda: q.act8_dequantize(q.Act8(None, None))):
        with pytest.raises(TypeError):
            call()
    assert act8.width(t, "X") == act8.width(q.Act8(t, t), "X") == 128 and act8.width(t[0], "X") == -1


@pytest.mark.gpu
def test_entry_points(q):
    bf = torch.bfloat16
    X, A, B = (torch.zeros(*s, dtype=bf, device="cuda") for s in ((8, 64), (64, 8), (8, 128)))
    w = q.quantize(torch.randn(64, 128, device="cuda").to(bf))
    args = (w, w, A, B, A, B, 1.0)
    dH = torch.zeros(8, 128, dtype=bf, device="cuda")
    _, saved = q.gated_forward(X, *args, save="bf16")
    y, f = torch.zeros(8, dtype=torch.int64, device="cuda"), torch.zeros(8, device="cuda")
    nothing = q.Act8(None, None)
    for call in (lambda: q.gated_forward(X, None, *args[1:]), lambda: q.gated_forward(X, w, dH, *args[2:]),
                 lambda: q.gated_forward(X, *args, saved=(dH, dH, X, X)),
                 lambda: q.gated_backward(dH, None, saved, *args), lambda: q.gated_backward(dH, nothing, saved, *args),
                 lambda: q.gated_backward(dH, X, q.GatedSaved(None, None, saved.Zg, saved.Zu), *args),
                 lambda: q.gated_backward(dH, X, saved, dH, *args[1:]),
                 lambda: q.linear_backward(dH, nothing, saved.Zg, w, A, B, 1.0),
                 lambda: q.linear_backward(dH, None, saved.Zg, w, A, B, 1.0, grad_dtype=bf),
                 lambda: q.linear_backward(dH, q.act8_quantize(X), saved.Zg, None, A, B, 1.0),
                 lambda: q.act8_dequantize(nothing), lambda: q.act8_quantize(X, out=(X, X)),
                 lambda: q.head_loss_forward(X, None, y), lambda: q.head_loss_forward(X, dH, y),
                 lambda: q.head_loss_forward(X, w, [0] * 8), lambda: q.head_loss_backward(f, X, f, None, y),
                 lambda: q.head_loss_backward(None, X, f, w, y)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("save", ["bf16", "int8"])
def test_empty_buffers_are_what_the_calls_take(q, save):
    bf = torch.bfloat16
    torch.manual_seed(3)
    X, A, B = (torch.randn(*s, device="cuda").to(bf) for s in ((40, 64), (64, 8), (8, 128)))
    w = q.quantize(torch.randn(64, 128, device="cuda").to(bf))
    args = (w, w, A, B, A, B, 0.5)
    H, want = q.gated_forward(X, *args, save=save)
    kept = q.GatedSaved.empty(40, 128, 8, save)
    H2, got = q.gated_forward(X, *args, saved=kept)
    assert got is kept and torch.equal(H, H2)

    def parts(s):
        return (s.G.codes, s.G.scales, s.U.codes, s.U.scales, s.Zg, s.Zu) if save == "int8" else (s.G, s.U, s.Zg, s.Zu)
    assert all(torch.equal(a, b) for a, b in zip(parts(want), parts(kept)))
    a = q.Act8.empty(40, 64)
    b = q.act8_quantize(X)
    assert q.act8_quantize(X, out=a) is a and torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
