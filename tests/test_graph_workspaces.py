"""Workspaces of captured calls: two graphs never share one, so that they may be
replayed at the same time, whichever stream they were captured on."""
import pytest
import torch


@pytest.fixture(scope="module")
def q():
    from tests.conftest import ensure_built
    ensure_built()
    import bit_nf4_quantized_pack_b200
    return bit_nf4_quantized_pack_b200


def test_a_capture_gets_buffers_of_its_own(q, monkeypatch):
    capturing = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type("S", (), {"cuda_stream": 11})())
    like = torch.empty(1)
    eager = q._workspace(None, "test", 512, like)
    assert q._workspace(None, "test", 300, like) is eager
    capturing[0] = True
    one, two = q._workspace(None, "test", 512, like), q._workspace(None, "test", 512, like)
    assert len({t.data_ptr() for t in (eager, one, two)}) == 3 and one.numel() >= 512
    # more than the cached one holds, and a purpose that was never called before
    assert q._workspace(None, "test", 4096, like).numel() >= 4096
    assert q._workspace(None, "never", 64, like).numel() >= 64
    assert q._workspace(eager, "test", 512, like) is eager and q._workspace(None, "test", 0, like) is None
    capturing[0] = False
    assert q._workspace(None, "test", 512, like) is eager


@pytest.mark.gpu
@pytest.mark.parametrize("rows,policy", [(8, "save"), (300, "save"), (300, "recompute"), (1500, "int8")])
def test_two_chains_captured_on_one_stream_and_replayed_at_once(q, rows, policy):
    from bit_nf4_quantized_pack_b200.chain import GatedLayer, HeadLoss, Layer, LinearChain
    torch.manual_seed(rows)

    def t(*shape, sigma=1.0):
        return (torch.randn(*shape, device="cuda") * sigma).to(torch.bfloat16)
    D, F, r = 512, 1344, 12           # the rank is padded: copies of A and Z in the workspaces
    layers = [Layer(q.quantize(t(D, D, sigma=0.05)), t(D, r, sigma=0.05), t(r, D, sigma=0.05), 2.0),
              GatedLayer(q.quantize(t(D, F, sigma=0.05)), q.quantize(t(D, F, sigma=0.05)), t(D, r, sigma=0.05),
                         t(r, F, sigma=0.05), t(D, r, sigma=0.05), t(r, F, sigma=0.05), 2.0),
              Layer(q.quantize(t(F, D, sigma=0.05)), t(F, r, sigma=0.05), t(r, D, sigma=0.05), 2.0)]
    head = HeadLoss(q.quantize(t(D, 640, sigma=0.1)), vocab=600)
    st = q.new_status()
    y = torch.randint(600, (rows,), device="cuda")
    xs = [t(rows, D) for _ in range(2)]

    def step(x):
        mean, dX, grads = LinearChain(layers, policy, head=head).loss_backward(x, y, status=st)
        w = q.quantize(x, double_quant=True, status=st)
        return [mean, dX, w.packed, w.s2, *(g for d in grads for g in d)]
    want = [[a.clone() for a in step(x)] for x in xs]
    side = torch.cuda.Stream()        # no call before its captures
    graphs = []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = step(x)
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, out), ref in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert q.status_sync(st) == (0, 0)
