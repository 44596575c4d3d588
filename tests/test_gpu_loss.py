"""The head loss on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

from inputs import synthetic as S
from oracle import loss as oracle
from tests._gpu_util import assert_close, to_dev, to_np
from tests._operators_util import HALF, SLACK, TINY, DecodedWeight, assert_within, gamma

pytestmark = pytest.mark.gpu
EXP = 2.0 ** -18    # the hardware's exponential, sums of up to a few thousand of them in fp32 included


def _q():
    import bit_nf4_quantized_pack_b200 as q
    return q


class Case:
    def __init__(self, M, K, vocab, kind, sigma=0.1, seed=21):
        N = -(-vocab // 64) * 64
        self.M, self.K, self.N, self.vocab = M, K, N, vocab
        self.w = DecodedWeight(S.normal(seed, M + K, 0, (K, N), sigma), kind)
        self.X = np.asarray(S.normal(seed, vocab, 1, (M, K), 1.0), np.float64)
        g = np.random.default_rng([seed, M, vocab])
        self.labels = g.integers(0, vocab, M)
        self.labels[g.random(M) < 0.15] = -100
        self.labels[0] = vocab - 1                # the last column that counts
        self.dloss = g.normal(size=M).astype(np.float32)
        self.t = (to_dev(self.X), self.w.dev, torch.from_numpy(self.labels).cuda())

    def bounds(self):
        W = self.w.hat[:, :self.vocab]
        logits = self.X @ W
        d = gamma(self.K) * (np.abs(self.X) @ np.abs(W))        # of each logit
        lse = oracle.head_loss_forward(self.X, self.w.hat, self.labels, self.vocab)[1]
        at = np.where(self.labels == -100, 0, self.labels)
        dl = d.max(1) + EXP + 2.0 ** -22 * np.abs(lse)
        dloss = dl + d[np.arange(self.M), at] + 2.0 ** -23 * np.abs(logits[np.arange(self.M), at])
        p = np.exp(logits - lse[:, None])
        s = p.copy()
        s[np.arange(self.M), at] -= 1
        scale = np.where(self.labels == -100, 0, np.abs(self.dloss.astype(np.float64)))[:, None]
        dP = scale * (HALF * np.abs(s) + p * (np.expm1(d + dl[:, None]) + EXP) + 2.0 ** -23)
        dX = oracle.head_loss_backward(self.dloss, self.X, self.w.hat, self.labels, self.vocab)
        err = dP @ np.abs(W).T + gamma(self.vocab + 64) * ((scale * np.abs(s)) @ np.abs(W).T) + HALF * np.abs(dX)
        return (lse, dl), dloss, (dX, err)


CASES = [  # M, K, vocab, weight
    (1, 64, 2, "dq"),
    (1, 64, 64, "absmax"),
    (3, 128, 65, "dq"),
    (33, 256, 1000, "dq"),
    (257, 192, 257, "int4"),
    (129, 64, 8190, "dq"),
    (520, 320, 511, "absmax"),
    (1030, 64, 640, "dq"),
]


@pytest.mark.parametrize("M,K,vocab,kind", CASES)
def test_loss_and_gradient(M, K, vocab, kind):
    q = _q()
    case = Case(M, K, vocab, kind)
    X, w, labels = case.t
    loss, lse = q.head_loss_forward(X, w, labels, vocab=vocab)
    ref_loss, ref_lse = oracle.head_loss_forward(case.X, case.w.hat, case.labels, vocab)
    (_, dl), dloss, (dX, err) = case.bounds()
    assert loss.dtype == lse.dtype == torch.float32
    assert_within("lse", to_np(lse), ref_lse, SLACK * dl + TINY)
    assert_within("loss", to_np(loss), ref_loss, SLACK * dloss + TINY)
    assert not to_np(loss)[case.labels == -100].any()
    got = q.head_loss_backward(torch.from_numpy(case.dloss).cuda(), X, lse, w, labels, vocab=vocab)
    assert_within("dX", to_np(got), dX, SLACK * err + TINY)
    assert_close("dX", to_np(got), dX)
    assert not to_np(got)[case.labels == -100].any()


def test_many_pieces():
    """Enough rows that the gradient runs over several pieces of the vocabulary
    (a piece holds about 2^26 elements), the last one ragged."""
    q = _q()
    M, K, vocab = 18000, 64, 8190
    case = Case(M, K, vocab, "dq", sigma=0.2)
    X, w, labels = case.t
    loss, lse = q.head_loss_forward(X, w, labels, vocab=vocab)
    dl = torch.from_numpy(case.dloss).cuda()
    got = q.head_loss_backward(dl, X, lse, w, labels, vocab=vocab)
    rows = np.r_[0:40, 8960:9000, 17960:18000]
    sub = Case.__new__(Case)
    sub.__dict__.update(case.__dict__, M=len(rows), X=case.X[rows], labels=case.labels[rows], dloss=case.dloss[rows])
    (ref_lse, dlse), dloss, (dX, err) = sub.bounds()
    assert_within("lse", to_np(lse)[rows], ref_lse, SLACK * dlse + TINY)
    # the pieces' sums meet in fp32: one more addition each
    assert_within("dX", to_np(got)[rows], dX, SLACK * err + TINY)
    # rows do not depend on their neighbours: the same rows alone
    i = torch.from_numpy(rows).cuda()
    l2, s2 = q.head_loss_forward(X[i].contiguous(), w, labels[i].contiguous(), vocab=vocab)
    assert torch.equal(l2, loss[i]) and torch.equal(s2, lse[i])


def test_sharp_and_flat_rows():
    """Logits of some hundreds (one token takes all the weight) and of zero."""
    q = _q()
    case = Case(40, 128, 500, "absmax", sigma=0.3)
    X = case.X.copy()
    X[::2] = S.f32_to_bf16_values((X[::2] * 40).astype(np.float32))
    X[1] = 0
    case.X = X
    Xt = to_dev(X)
    case.labels[2] = int(np.argmax(X[2] @ case.w.hat[:, :500]))       # a loss near zero
    labels = torch.from_numpy(case.labels).cuda()
    loss, lse = q.head_loss_forward(Xt, case.t[1], labels, vocab=500)
    (ref, dl), dloss, (dX, err) = case.bounds()
    assert_within("lse", to_np(lse), ref, SLACK * dl + TINY)
    assert_within("loss", to_np(loss), oracle.head_loss_forward(X, case.w.hat, case.labels, 500)[0], SLACK * dloss + TINY)
    assert abs(float(lse[1]) - np.log(500)) < 1e-5
    got = q.head_loss_backward(torch.from_numpy(case.dloss).cuda(), Xt, lse, case.t[1], labels, vocab=500)
    assert_within("dX", to_np(got), dX, SLACK * err + TINY)


def test_labels_outside_the_vocabulary_are_reported():
    q = _q()
    case = Case(10, 64, 100, "dq")
    X, w, labels = case.t
    for bad in (100, 127, 128, -1, 2 ** 40):
        y = labels.clone()
        y[3] = bad
        st = q.new_status()
        loss, lse = q.head_loss_forward(X, w, y, vocab=100, status=st)
        assert q.status_sync(st)[0] == 1
        assert loss[3] == 0 and torch.isfinite(lse).all()
        dX = q.head_loss_backward(torch.ones(10, device="cuda"), X, lse, w, y, vocab=100, status=st)
        assert not dX[3].any() and torch.isfinite(dX).all()
    # another ignore_index, one inside the vocabulary
    y = labels.clone()
    y[:] = 7
    loss, _ = q.head_loss_forward(X, w, y, vocab=100, ignore_index=7)
    assert not loss.any()


def test_padding_columns_do_not_count():
    """The head's columns behind the vocabulary change nothing, whatever they hold."""
    q = _q()
    M, K, vocab, N = 50, 64, 300, 576
    W = S.normal(3, 4, 0, (K, N), 0.1)
    W2 = W.copy()
    W2[:, 320:] = 5.0                     # whole blocks behind the vocabulary's last one
    X, labels = to_dev(S.normal(3, 4, 1, (M, K), 1.0)), torch.arange(M, device="cuda")
    dl = torch.ones(M, device="cuda")
    outs = []
    for w in (q.quantize(to_dev(W), double_quant=False), q.quantize(to_dev(W2), double_quant=False)):
        loss, lse = q.head_loss_forward(X, w, labels, vocab=vocab)
        outs.append((loss, lse, q.head_loss_backward(dl, X, lse, w, labels, vocab=vocab)))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_outputs_stay_inside():
    q = _q()
    case = Case(77, 192, 200, "dq")
    X, w, labels = case.t
    pad = 64

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        big = torch.full((n + 2 * pad,), 5, dtype=dtype, device="cuda")
        return big, big[pad:pad + n].view(shape)
    a, b, c = guarded((77,), torch.float32), guarded((77,), torch.float32), guarded((77, 192), torch.bfloat16)
    q.head_loss_forward(X, w, labels, vocab=200, loss=a[1], lse=b[1])
    q.head_loss_backward(torch.ones(77, device="cuda"), X, b[1], w, labels, vocab=200, dX=c[1])
    for big, t in (a, b, c):
        assert (big[:pad] == 5).all() and (big[pad + t.numel():] == 5).all() and (t != 5).any()
