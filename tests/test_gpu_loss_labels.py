"""Labels outside the vocabulary are a device error of the backward too, which
may run with a status word that the forward never saw."""
import pytest
import torch

from inputs import synthetic as S
from tests._gpu_util import to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,vocab,row", [(10, 100, 3), (300, 700, 299), (1, 64, 0)])
def test_backward_reports_labels_outside_the_vocabulary(M, vocab, row):
    import bit_nf4_quantized_pack_b200 as q
    N = -(-vocab // 64) * 64
    w = q.quantize(to_dev(S.normal(61, M, 0, (64, N), 0.1)))
    X, dl = to_dev(S.normal(61, M, 1, (M, 64), 1.0)), torch.ones(M, device="cuda")
    good = torch.arange(M, device="cuda") % vocab
    good[0] = vocab - 1
    loss, lse = q.head_loss_forward(X, w, good, vocab=vocab)
    st = q.new_status()
    want = q.head_loss_backward(dl, X, lse, w, good, vocab=vocab, status=st)
    assert q.status_sync(st) == (0, 0)
    for bad in (vocab, N, -1, 2 ** 40, -2 ** 40):
        y = good.clone()
        y[row] = bad
        st = q.new_status()
        dX = q.head_loss_backward(dl, X, lse, w, y, vocab=vocab, status=st)
        assert q.status_sync(st) == (1, 2)
        assert not dX[row].any()
        rest = [i for i in range(M) if i != row]
        assert torch.equal(dX[rest], want[rest])
        with pytest.raises(q.QLoRAError):
            q.head_loss_backward(dl, X, lse, w, y, vocab=vocab)
        # the same label left out on purpose is none
        st = q.new_status()
        again = q.head_loss_backward(dl, X, lse, w, y, vocab=vocab, ignore_index=bad, status=st)
        assert q.status_sync(st) == (0, 0) and torch.equal(again, dX)
