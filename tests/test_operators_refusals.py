"""What the gated block, the 8-bit checkpoints and the head loss refuse, before
any device work: the C ABI's host validation, and the wrappers' checks."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from tests.conftest import ensure_built
    ensure_built()
    from bit_nf4_quantized_pack_b200 import _lib
    return _lib


@pytest.fixture(scope="module")
def q(L):
    import bit_nf4_quantized_pack_b200
    return bit_nf4_quantized_pack_b200


P = 4096           # an aligned address that is never read
BIG = 1 << 40      # workspace bytes


def state(L, numel, **kw):
    st = L.NF4StateC(numel, 64, 0, 256, 0, P, P, P, P, P)
    for k, v in kw.items():
        setattr(st, k, v)
    return st


def saved(L, **kw):
    d = dict(G=P, U=P, Zg=P, Zu=P)
    d.update(kw)
    return L.GatedSavedC(**d)


def fwd(L, M=8, K=64, N=128, r=8, X=P, wg=None, wu=None, Ag=P, Bg=P, Au=P, Bu=P, c=1.0, act=0, H=P, kept=None,
        ws=P, n=BIG):
    wg = wg if wg is not None else state(L, K * N)
    wu = wu if wu is not None else state(L, K * N)
    return L.lib.qlora_gated_fwd(M, K, N, r, X, C.byref(wg), C.byref(wu), Ag, Bg, Au, Bu, c, act, H,
                                 C.byref(kept) if kept is not None else None, ws, n, None, None)


def test_gated_forward(L):
    bad, uns = L.QLORA_ERR_INVALID_ARG, L.QLORA_ERR_UNSUPPORTED
    for kw in (dict(M=0), dict(X=None), dict(X=P + 2), dict(Ag=None), dict(Bg=P + 8), dict(Au=None), dict(Bu=None),
               dict(H=None), dict(H=P + 4), dict(c=float("nan")), dict(c=float("inf")), dict(act=2), dict(act=-1),
               dict(ws=None), dict(n=16), dict(ws=P + 1), dict(wg=state(L, 64)), dict(wu=state(L, 64)),
               dict(wu=state(L, 64 * 128, packed=None)), dict(wg=state(L, 64 * 128, absmax=None)),
               dict(wg=state(L, 64 * 128, blocksize=128)), dict(wg=state(L, 64 * 128, codebook=2))):
        assert fwd(L, **kw) == bad, kw
    for kw in (dict(K=65), dict(N=100), dict(r=0), dict(r=65), dict(M=(1 << 30) + 1), dict(M=1 << 29, N=1 << 10),
               dict(wu=state(L, 64 * 128, codebook=1, double_quant=1))):
        assert fwd(L, **kw) == uns, kw
    # what the forward keeps: Z, and g and u in exactly one form
    for kw in (dict(Zg=None), dict(Zu=P + 2), dict(U=None), dict(G=None, U=None), dict(G8=P),
               dict(G=None, U=None, G8=P, U8=P, G_scales=P), dict(G=P + 2)):
        assert fwd(L, kept=saved(L, **kw)) == bad, kw


def test_gated_backward(L):
    bad = L.QLORA_ERR_INVALID_ARG
    w = state(L, 64 * 128)
    a8 = L.Act8C(8, 64, P, P)

    def bwd(X=P, X8=None, kept=None, dt=1, dX=P, dAg=P, dBu=P, dH=P, n=BIG, r=8):
        kept = kept if kept is not None else saved(L)
        return L.lib.qlora_gated_bwd(8, 64, 128, r, dH, X, C.byref(X8) if X8 is not None else None, C.byref(kept),
                                     C.byref(w), C.byref(w), P, P, P, P, 1.0, 0, dX, dAg, P, P, dBu, dt, P, n, None,
                                     None)
    for kw in (dict(X=None), dict(X8=a8), dict(X=P + 2), dict(dt=2), dict(dX=None), dict(dAg=P + 4), dict(dBu=None),
               dict(dH=None), dict(n=100), dict(kept=saved(L, G=None)), dict(X=None, X8=L.Act8C(9, 64, P, P)),
               dict(X=None, X8=L.Act8C(8, 128, P, P)), dict(X=None, X8=L.Act8C(8, 64, None, P)),
               dict(X=None, X8=L.Act8C(8, 64, P, P + 2))):
        assert bwd(**kw) == bad, kw
    assert bwd(r=65) == L.QLORA_ERR_UNSUPPORTED
    assert L.lib.qlora_gated_bwd(8, 64, 128, 8, P, P, None, None, C.byref(w), C.byref(w), P, P, P, P, 1.0, 0, P, P, P,
                                 P, P, 1, P, BIG, None, None) == bad


def test_linear_backward_from_codes(L):
    bad = L.QLORA_ERR_INVALID_ARG
    w = state(L, 64 * 128)

    def bwd(X=None, X8=L.Act8C(8, 64, P, P), Zc=P, dt=0, dA=P, n=BIG, c=1.0):
        return L.lib.qlora_linear_bwd_act8(8, 64, 128, 8, P, X, C.byref(X8) if X8 is not None else None, Zc,
                                           C.byref(w), P, P, c, P, dA, P, dt, P, n, None, None)
    for kw in (dict(X=P), dict(X8=None), dict(Zc=None), dict(dt=7), dict(dA=None), dict(n=8), dict(c=float("nan")),
               dict(X8=L.Act8C(7, 64, P, P)), dict(Zc=P + 2)):
        assert bwd(**kw) == bad, kw


def test_act8(L):
    bad, uns = L.QLORA_ERR_INVALID_ARG, L.QLORA_ERR_UNSUPPORTED
    lib = L.lib
    for a in (L.Act8C(0, 64, P, P), L.Act8C(4, 0, P, P), L.Act8C(4, 64, None, P), L.Act8C(4, 64, P, None),
              L.Act8C(4, 64, P + 4, P)):
        assert lib.qlora_act8_quantize(P, C.byref(a), None, None) == bad
        assert lib.qlora_act8_dequantize(C.byref(a), P, None) == bad
    assert lib.qlora_act8_quantize(P, None, None, None) == bad
    for a in (L.Act8C(4, 96, P, P), L.Act8C(1 << 33, 64, P, P)):
        assert lib.qlora_act8_quantize(P, C.byref(a), None, None) == uns
    ok = L.Act8C(4, 64, P, P)
    assert lib.qlora_act8_quantize(None, C.byref(ok), None, None) == bad
    assert lib.qlora_act8_quantize(P + 2, C.byref(ok), None, None) == bad
    assert lib.qlora_act8_dequantize(C.byref(ok), None, None) == bad


def test_head_loss(L):
    bad, uns = L.QLORA_ERR_INVALID_ARG, L.QLORA_ERR_UNSUPPORTED
    w = state(L, 64 * 128)

    def fwd_(M=8, K=64, N=128, vocab=100, X=P, y=P, loss=P, lse=P, n=BIG, ws=P):
        return L.lib.qlora_head_loss_fwd(M, K, N, vocab, X, C.byref(w), y, -100, loss, lse, ws, n, None, None)

    def bwd_(M=8, K=64, N=128, vocab=100, X=P, y=P, dl=P, lse=P, dX=P, n=BIG):
        return L.lib.qlora_head_loss_bwd(M, K, N, vocab, dl, X, lse, C.byref(w), y, -100, dX, P, n, None, None)
    for kw in (dict(M=0), dict(vocab=0), dict(vocab=129), dict(X=None), dict(y=None), dict(y=P + 4), dict(lse=None),
               dict(n=8), dict(N=64)):
        assert fwd_(**kw) == bad, kw
        assert bwd_(**kw) == bad, kw
    assert fwd_(loss=P + 2) == bad and fwd_(ws=None) == bad
    assert bwd_(dl=None) == bad and bwd_(dX=P + 2) == bad
    for kw in (dict(K=63), dict(N=130), dict(M=1 << 30, N=1 << 20)):
        assert fwd_(**kw) == uns and bwd_(**kw) == uns


def test_workspace_sizes(L):
    lib = L.lib
    assert lib.qlora_gated_fwd_workspace_size(8, 65, 64, 8) == 0
    assert lib.qlora_gated_bwd_workspace_size(8, 64, 64, 0) == 0
    assert lib.qlora_head_loss_fwd_workspace_size(0, 64, 64) == 0
    # dG and dU are in the backward's
    assert lib.qlora_gated_bwd_workspace_size(300, 64, 128, 8) >= 2 * 300 * 128 * 2
    # a row's pair of statistics per 256 columns
    assert lib.qlora_head_loss_fwd_workspace_size(10, 64, 1024) >= 10 * 4 * 8
    # pieces: about 2^26 elements of P however large the vocabulary, and the fp32 sums
    big = lib.qlora_head_loss_bwd_workspace_size(4096, 4096, 1 << 20)
    assert 4096 * 4096 * 4 < big <= 4096 * 4096 * 4 + (1 << 27) + 4096 * 512 * 2
    # few rows: one slot per CTA and group at most
    assert lib.qlora_gated_fwd_workspace_size(1, 4096, 11008, 16) < 1 << 20


def cpu_weight(q, K=64, N=128):
    n1 = K * N // 64
    return q.NF4Weight((K, N), False, torch.zeros(K * N // 2, dtype=torch.uint8), torch.zeros(n1))


def test_wrappers_refuse_cpu_tensors_and_wrong_types(q):
    b = torch.zeros(8, 64, dtype=torch.bfloat16)
    w = cpu_weight(q)
    A, B = torch.zeros(64, 8, dtype=torch.bfloat16), torch.zeros(8, 128, dtype=torch.bfloat16)
    for call in (lambda: q.act8_quantize(b), lambda: q.act8_dequantize(q.Act8(b, b)),
                 lambda: q.act8_dequantize(b), lambda: q.gated_forward(b, w, w, A, B, A, B, 1.0),
                 lambda: q.gated_backward(b, b, None, w, w, A, B, A, B, 1.0),
                 lambda: q.head_loss_forward(b, w, torch.zeros(8, dtype=torch.int64)),
                 lambda: q.head_loss_backward(b, b, b, w, b),
                 lambda: q.linear_backward(b, q.Act8(b, b), None, w, A, B, 1.0),
                 lambda: q.linear_backward(b, b, None, w, A, B, 1.0, grad_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_wrappers_refuse_wrong_shapes_and_short_buffers(q):
    bf = torch.bfloat16

    def t(*shape, dtype=bf):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    X, A, B = t(8, 64), t(64, 8), t(8, 128)
    w = q.quantize(torch.randn(64, 128, device="cuda").to(bf))
    args = [w, w, A, B, A, B, 1.0]
    H, saved_ = q.gated_forward(X, *args, save="bf16")
    dH = t(8, 128)
    short = q.NF4Weight((64, 128), True, w.packed[:-16], code8=w.code8, s2=w.s2, offset=w.offset)
    other = q.quantize(torch.randn(128, 64, device="cuda").to(bf))
    for call in (lambda: q.gated_forward(t(8, 128), *args), lambda: q.gated_forward(t(8), *args),
                 lambda: q.gated_forward(X, short, *args[1:]), lambda: q.gated_forward(X, w, other, *args[2:]),
                 lambda: q.gated_forward(X, w, w, A, t(4, 128), A, B, 1.0),
                 lambda: q.gated_forward(X, w, w, A, B, t(64, 4), B, 1.0),
                 lambda: q.gated_forward(X, *args, act="tanh"), lambda: q.gated_forward(X, *args, save="fp8"),
                 lambda: q.gated_forward(X, *args, H=t(8, 64)),
                 lambda: q.gated_forward(X, *args, workspace=t(16, dtype=torch.uint8)),
                 lambda: q.gated_backward(t(7, 128), X, saved_, *args),
                 lambda: q.gated_backward(dH, t(8, 128), saved_, *args),
                 lambda: q.gated_backward(t(8, 64), X, saved_, *args),
                 lambda: q.gated_backward(dH, X, q.GatedSaved(saved_.G, saved_.U, saved_.Zg[:4], saved_.Zu), *args),
                 lambda: q.gated_backward(dH, X, saved_, *args, dAg=t(8, 64, dtype=torch.float32)),
                 lambda: q.act8_quantize(X, out=q.Act8(t(8, 64, dtype=torch.int8), t(8, 2, dtype=torch.float32))),
                 lambda: q.act8_dequantize(q.Act8(t(8, 64, dtype=torch.int8), t(7, 1, dtype=torch.float32))),
                 lambda: q.linear_backward(dH, q.act8_quantize(X), None, w, A, B, 1.0),
                 lambda: q.linear_backward(dH, q.act8_quantize(t(9, 64)), t(8, 8), w, A, B, 1.0),
                 lambda: q.head_loss_forward(X, w, torch.zeros(7, dtype=torch.int64, device="cuda")),
                 lambda: q.head_loss_forward(X, w, torch.zeros(8, dtype=torch.int64, device="cuda"), vocab=129),
                 lambda: q.head_loss_backward(t(7, dtype=torch.float32), X, t(8, dtype=torch.float32), w,
                                              torch.zeros(8, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: q.gated_forward(X.float(), *args), lambda: q.gated_forward(t(64, 8).t(), *args),
                 lambda: q.gated_forward(X, w, w, A.float(), B, A, B, 1.0),
                 lambda: q.gated_backward(dH, X, saved_, *args, dX=t(8, 64, dtype=torch.float32)),
                 lambda: q.gated_backward(dH, X, (H, H), *args),
                 lambda: q.head_loss_forward(X, w, torch.zeros(8, dtype=torch.int32, device="cuda")),
                 lambda: q.act8_quantize(t(8, 128)[:, ::2]),
                 lambda: q.act8_quantize(X, status=torch.zeros(1, dtype=torch.int32)),
                 lambda: q.gated_forward(X, *args, status=t(1))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: q.act8_quantize(t(8, 96)), lambda: q.act8_quantize(t(0, 64)),
                 lambda: q.gated_forward(t(0, 64), *args),
                 lambda: q.gated_forward(X, w, w, A, B, A, B, float("nan"))):
        with pytest.raises(q.QLoRAError):
            call()
