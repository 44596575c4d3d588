"""The backwards that run dA and dB on the library's own stream, beside other
captures: a captured backward takes that stream into its capture until the
capture ends, and a backward elsewhere must then do without it."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
M, K, N, R = 1030, 1088, 11008, 16        # M K N > 1e10: all of these run beside dX


def _q():
    import bit_nf4_quantized_pack_b200 as q
    return q


def bf16(g, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)


class Call:
    """One backward with all its buffers given, so that it allocates nothing."""

    def __init__(self, kind, seed):
        q = _q()
        g = torch.Generator(device="cuda").manual_seed(seed)
        X, A, B = bf16(g, M, K), bf16(g, K, R, sigma=0.02), bf16(g, R, N, sigma=0.02)
        w = q.quantize(bf16(g, K, N, sigma=0.02))
        dY = bf16(g, M, N)
        self.st = q.new_status()
        lib = q.lib
        empty = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        dX = empty(M, K, dtype=torch.bfloat16)
        if kind == "gated":
            wu = q.quantize(bf16(g, K, N, sigma=0.02))
            args = (w, wu, A, B, A, B, 2.0)
            saved = q.gated_forward(X, *args, save="bf16")[1]
            out = dict(dX=dX, dAg=empty(K, R), dBg=empty(R, N), dAu=empty(K, R), dBu=empty(R, N))
            ws = empty(lib.qlora_gated_bwd_workspace_size(M, K, N, R), dtype=torch.uint8)
            self.run = lambda: q.gated_backward(dY, X, saved, *args, status=self.st, workspace=ws, **out)
        else:
            Zc = q.linear_forward(X, w, A, B, 2.0)[1]
            out = dict(dX=dX, dA=empty(K, R), dB=empty(R, N))
            ws = empty(lib.qlora_linear_bwd_workspace_size(M, K, N, R), dtype=torch.uint8)
            x = q.act8_quantize(X) if kind == "act8" else X
            self.run = lambda: q.linear_backward(dY, x, Zc, w, A, B, 2.0, status=self.st, workspace=ws, **out)
        self.out = out
        self.run()
        torch.cuda.synchronize()
        self.want = {n: t.clone() for n, t in out.items()}

    def check(self):
        torch.cuda.synchronize()
        assert _q().status_sync(self.st) == (0, 0)
        for n, t in self.out.items():
            assert torch.equal(t, self.want[n]), n

    def clear(self):
        for t in self.out.values():
            t.fill_(float("nan"))
        torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["gated", "act8", "linear"])
def test_other_stream_and_graph_give_the_same_bits(kind):
    c = Call(kind, 71)
    side = torch.cuda.Stream()
    c.clear()
    with torch.cuda.stream(side):
        c.run()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        c.run()
    for _ in range(2):
        c.clear()
        g.replay()
        c.check()


@pytest.mark.parametrize("captured,eager,default", [("gated", "linear", False), ("linear", "gated", False),
                                                    ("act8", "act8", False), ("gated", "gated", True)])
def test_eager_backward_while_another_stream_is_capturing(captured, eager, default):
    a, b = Call(captured, 72), Call(eager, 73)
    mine, other = torch.cuda.Stream(), torch.cuda.default_stream() if default else torch.cuda.Stream()
    a.clear()
    b.clear()
    failed = []

    def work():
        try:
            with torch.cuda.stream(other):
                b.run()
        except Exception as e:             # noqa: BLE001  (reported by the test's own thread)
            failed.append(e)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=mine, capture_error_mode="thread_local"):
        a.run()                            # the library's stream is part of this capture from here on
        t = threading.Thread(target=work)
        t.start()
        t.join()
        a.run()
    assert not failed, failed
    b.check()
    g.replay()
    a.check()
    # and afterwards both as before
    for c in (a, b):
        c.clear()
        c.run()
        c.check()
