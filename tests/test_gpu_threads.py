"""Every entry point as the first CUDA work of a thread, with all buffers given,
so that nothing before the library's call has made the device's context current
there."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
K, N, R = 256, 320, 16


def bf16(*shape, sigma=1.0):
    return (torch.randn(*shape, device="cuda") * sigma).to(torch.bfloat16)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_first_call_of_a_thread(M):
    import bit_nf4_quantized_pack_b200 as q
    torch.manual_seed(M)
    w = q.quantize(bf16(K, N, sigma=0.05))
    X, dY, A, B = bf16(M, K), bf16(M, N), bf16(K, R, sigma=0.05), bf16(R, N, sigma=0.05)
    st = q.new_status()
    y = torch.arange(M, device="cuda")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    block = (w, w, A, B, A, B, 2.0)
    H, saved = q.gated_forward(X, *block, save="bf16")
    Zc = q.linear_forward(X, w, A, B, 2.0)[1]
    loss, lse = q.head_loss_forward(X, w, y)
    a8, packed = q.act8_quantize(X), torch.empty_like(w.packed)
    again = q.NF4Weight((K, N), True, packed, code8=torch.empty_like(w.code8), s2=torch.empty_like(w.s2),
                        offset=torch.empty_like(w.offset))
    Wd = q.dequantize(w)

    def new(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    b = torch.bfloat16
    kw = dict(status=st, workspace=ws)
    calls = {
        "quantize": lambda o: (q.quantize(Wd, out=again, **kw), [again.packed, again.s2])[1],
        "dequantize": lambda o: [q.dequantize(w, out=o[0], status=st)],
        "merge": lambda o: [q.merge(w, A, B, 1.0, out=o[0], status=st)],
        "linear_forward": lambda o: q.linear_forward(X, w, A, B, 2.0, Y=o[0], Zc=o[1], **kw),
        "linear_backward": lambda o: q.linear_backward(dY, X, Zc, w, A, B, 2.0, dX=o[0], dA=o[1], dB=o[2], **kw),
        "from codes": lambda o: q.linear_backward(dY, a8, Zc, w, A, B, 2.0, dX=o[0], dA=o[1], dB=o[2], **kw),
        "act8_quantize": lambda o: [q.act8_quantize(X, out=q.Act8(*o), status=st).codes, o[1]],
        "act8_dequantize": lambda o: [q.act8_dequantize(a8, out=o[0])],
        "gated_forward": lambda o: [q.gated_forward(X, *block, H=o[0], **kw)[0]],
        "gated_backward": lambda o: q.gated_backward(dY, X, saved, *block, dX=o[0], dAg=o[1], dBg=o[2], dAu=o[3],
                                                     dBu=o[4], **kw),
        "head_loss_forward": lambda o: q.head_loss_forward(X, w, y, loss=o[0], lse=o[1], **kw),
        "head_loss_backward": lambda o: [q.head_loss_backward(loss, X, lse, w, y, dX=o[0], **kw)],
    }
    outs = {
        "quantize": lambda: [], "dequantize": lambda: [new(K, N, dtype=b)], "merge": lambda: [new(K, N, dtype=b)],
        "linear_forward": lambda: [new(M, N, dtype=b), new(M, R, dtype=b)],
        "linear_backward": lambda: [new(M, K, dtype=b), new(K, R), new(R, N)],
        "from codes": lambda: [new(M, K, dtype=b), new(K, R), new(R, N)],
        "act8_quantize": lambda: [new(M, K, dtype=torch.int8), new(M, K // 64)],
        "act8_dequantize": lambda: [new(M, K, dtype=b)],
        "gated_forward": lambda: [new(M, N, dtype=b)],
        "gated_backward": lambda: [new(M, K, dtype=b), new(K, R), new(R, N), new(K, R), new(R, N)],
        "head_loss_forward": lambda: [new(M), new(M)], "head_loss_backward": lambda: [new(M, K, dtype=b)],
    }
    failed = {}
    for name, call in calls.items():
        want = [t.clone() for t in call(outs[name]())]
        o = outs[name]()
        torch.cuda.synchronize()
        got = []

        def work():
            try:
                got.extend(call(o))
            except Exception as e:         # noqa: BLE001  (reported below)
                failed[name] = e
        t = threading.Thread(target=work)
        t.start()
        t.join()
        torch.cuda.synchronize()
        if name not in failed:
            assert all(torch.equal(x, z) for x, z in zip(got, want)), name
    assert not failed, failed
    assert q.status_sync(st) == (0, 0)
