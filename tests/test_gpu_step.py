"""The gated block, its neighbours and the head loss run together, as a
training step uses them: gated block -> down projection -> head -> loss, and
back, under the three saved-activation policies, eager, on another stream and
replayed from a CUDA graph."""
import numpy as np
import pytest
import torch

from inputs import synthetic as S
from oracle import gated as gated_oracle
from oracle import loss as loss_oracle
from oracle.linear import lora_backward, lora_forward
from tests._gpu_util import assert_close, to_dev, to_np
from tests._operators_util import DecodedWeight, GatedCase

pytestmark = pytest.mark.gpu
M, K, N, R, VOCAB = 150, 192, 320, 12, 300


def _q():
    import bit_nf4_quantized_pack_b200 as q
    return q


class Step:
    def __init__(self, seed=31, rows=M):
        from bit_nf4_quantized_pack_b200.chain import GatedLayer, HeadLoss, Layer
        self.case = GatedCase(seed, rows, K, N, R, ("dq", "absmax"))
        self.down = DecodedWeight(S.normal(seed, 50, 0, (N, K), 0.05), "dq")
        self.headw = DecodedWeight(S.normal(seed, 51, 0, (K, 320), 0.1), "dq")
        self.A, self.B = S.normal(seed, 52, 2, (N, R), 0.05), S.normal(seed, 52, 3, (R, K), 0.05)
        self.labels = np.random.default_rng(seed).integers(0, VOCAB, rows)
        self.labels[::7] = -100
        c, t = self.case, self.case.t
        self.layers = [GatedLayer(c.wg.dev, c.wu.dev, t["Ag"], t["Bg"], t["Au"], t["Bu"], c.c),
                       Layer(self.down.dev, to_dev(self.A), to_dev(self.B), 2.0)]
        self.head = HeadLoss(self.headw.dev, vocab=VOCAB)
        self.X, self.y = t["X"], torch.from_numpy(self.labels).cuda()

    def chain(self, policy):
        from bit_nf4_quantized_pack_b200.chain import LinearChain
        return LinearChain(self.layers, policy, head=self.head)


def flat(mean, dX, grads):
    return [mean, dX, *(t for g in grads for t in g)]


def test_step_against_the_oracle():
    """Every layer against the oracle on what that layer received."""
    s = Step()
    ch = s.chain("save")
    mean, dX, grads = ch.loss_backward(s.X, s.y)
    h = ch._inputs[1]                                       # the down projection's input
    c = s.case
    H = gated_oracle.gated_forward(c.host["X"], c.wg.hat, c.wu.hat, c.host["Ag"], c.host["Bg"], c.host["Au"],
                                   c.host["Bu"], c.c, "silu")[0]
    assert_close("H", to_np(h), H)
    A, B = (np.asarray(v, np.float64) for v in (s.A, s.B))
    Y, _ = lora_forward(to_np(h), s.down.hat, A, B, 2.0)
    out = to_np(ch.forward(s.X))
    assert_close("Y", out, Y)
    counted = s.labels != -100
    lo, _ = loss_oracle.head_loss_forward(out, s.headw.hat, s.labels, VOCAB)
    assert abs(float(mean) - lo.sum() / counted.sum()) <= 1e-5 * abs(lo.sum() / counted.sum())
    dY = loss_oracle.head_loss_backward(counted / counted.sum(), out, s.headw.hat, s.labels, VOCAB)
    # the device's own dY (bf16) for what is behind it
    dYd = s.head.backward(ch.forward(s.X), s.head.forward(ch.forward(s.X), s.y)[2], s.y)
    assert_close("dY", to_np(dYd), dY)
    dH, dA, dB = lora_backward(to_np(dYd), to_np(h), s.down.hat, A, B, 2.0)
    assert_close("dA", to_np(grads[1][0]), dA)
    assert_close("dB", to_np(grads[1][1]), dB)
    q = _q()
    dHd = q.linear_backward(dYd, h, ch._zc[1], s.down.dev, s.layers[1].A, s.layers[1].B, 2.0)[0]
    assert_close("dH", to_np(dHd), dH)
    kept = ch._zc[0]
    ref = gated_oracle.gated_backward(to_np(dHd), c.host["X"], to_np(kept.G), to_np(kept.U), c.wg.hat, c.wu.hat,
                                      c.host["Ag"], c.host["Bg"], c.host["Au"], c.host["Bu"], c.c, "silu")
    for n, got, want in zip(("dX", "dAg", "dBg", "dAu", "dBu"), (dX, *grads[0]), ref):
        assert_close(n, to_np(got), want)


@pytest.mark.parametrize("rows", [1, 16, M, 300])
def test_policies(rows):
    """recompute gives the bits of save; int8 gives the bits of the same calls
    on what its checkpoints stand for, and gradients near save's."""
    q = _q()
    s = Step(rows=rows)
    outs = {p: flat(*s.chain(p).loss_backward(s.X, s.y)) for p in ("save", "recompute", "int8")}
    for a, b in zip(outs["save"], outs["recompute"]):
        assert torch.equal(a, b)
    assert torch.equal(outs["save"][0], outs["int8"][0])            # the forward does not see the policy
    for a, b in zip(outs["save"][1:], outs["int8"][1:]):
        # 1 % of a block's largest value at most per kept element (half of 1 / 127,
        # two bf16 roundings), in sums over many
        assert float((a.double() - b.double()).norm()) <= 0.02 * float(a.double().norm()) + 1e-30
    ch = s.chain("int8")
    ch.loss_backward(s.X, s.y)
    assert isinstance(ch._inputs[0], q.Act8) and isinstance(ch._zc[0].G, q.Act8)


def test_small_steps_of_the_adapters_lower_the_loss_as_their_gradients_say():
    """The directional difference of the mean loss along the adapters'
    gradients, in fp64 through the oracle, against their norm."""
    s = Step(seed=33)
    mean, dX, grads = s.chain("save").loss_backward(s.X, s.y)
    c = s.case
    params = [c.host["Ag"], c.host["Bg"], c.host["Au"], c.host["Bu"], np.asarray(s.A, np.float64),
              np.asarray(s.B, np.float64)]
    G = [to_np(t) for t in (*grads[0], *grads[1])]
    counted = s.labels != -100

    def value(p):
        H = gated_oracle.gated_forward(c.host["X"], c.wg.hat, c.wu.hat, *p[:4], c.c, "silu")[0]
        Y = lora_forward(H, s.down.hat, p[4], p[5], 2.0)[0]
        return loss_oracle.head_loss_forward(Y, s.headw.hat, s.labels, VOCAB)[0].sum() / counted.sum()
    h = 1e-5
    slope = (value([p + h * g for p, g in zip(params, G)]) - value([p - h * g for p, g in zip(params, G)])) / (2 * h)
    norm = sum((g * g).sum() for g in G)
    # bf16 roundings of the activations and of dG, dU, dZ on the way: 2^-8 each
    # at most, about ten of them
    assert abs(slope - norm) <= 10 * 2.0 ** -8 * norm


def test_other_stream_and_graph_replay():
    s = Step(rows=200)
    ch = s.chain("int8")
    st = _q().new_status()
    want = [t.clone() for t in flat(*ch.loss_backward(s.X, s.y, status=st))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = flat(*ch.loss_backward(s.X, s.y, status=st))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = s.X.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        out = flat(*ch.loss_backward(x, s.y, status=st))
    for scale in (1, 2):                       # the captured input takes new values
        x.copy_((s.X.float() * scale).to(torch.bfloat16))
        ref = [t.clone() for t in flat(*ch.loss_backward(x, s.y, status=st))]
        torch.cuda.synchronize()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert _q().status_sync(st)[0] == 0


@pytest.mark.parametrize("rows", [8, 150])
def test_two_graphs_at_once(rows):
    """Graphs captured on one stream and replayed at the same time on two: each
    has workspaces of its own."""
    q = _q()
    s = Step(rows=rows)
    st = q.new_status()

    def body(x):
        H, saved = q.gated_forward(x, *s.case.args, save="int8", status=st)
        grads = q.gated_backward(s.case.t["dH"], q.act8_quantize(x, status=st), saved, *s.case.args, status=st)
        loss, lse = q.head_loss_forward(grads[0], s.headw.dev, s.y, vocab=VOCAB, status=st)
        d = q.head_loss_backward(loss, grads[0], lse, s.headw.dev, s.y, vocab=VOCAB, status=st)
        return [H, *grads, loss, lse, d]
    xs = [s.X.clone(), (s.X.float() * 2).to(torch.bfloat16)]
    want = [[t.clone() for t in body(x)] for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            out = body(x)
        graphs.append((g, out))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for (g, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for (_, out), ref in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert q.status_sync(st)[0] == 0


def test_two_calls_at_once_on_two_streams():
    q = _q()
    s = Step(rows=16)
    t = Step(seed=40, rows=300)
    want = [q.gated_forward(x.X, *x.case.args)[0].clone() for x in (s, t)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for stream, x in zip(streams, (s, t)):
            with torch.cuda.stream(stream):
                outs.append(q.gated_forward(x.X, *x.case.args, status=q.new_status())[0])
    torch.cuda.synchronize()
    for i, H in enumerate(outs):
        assert torch.equal(H, want[i % 2])
