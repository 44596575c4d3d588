"""LinearChain's layers on the CPU: what a chain accepts and refuses before any
device work."""
from types import SimpleNamespace

import pytest


@pytest.fixture(scope="module")
def chain():
    from tests.conftest import ensure_built
    ensure_built()
    from bit_nf4_quantized_pack_b200 import chain
    return chain


def weight(K, N):
    return SimpleNamespace(shape=(K, N))


def linear(K, N):
    return SimpleNamespace(w=weight(K, N), A=None, B=None, c=1.0)


def gated(chain, K, N):
    return chain.GatedLayer(weight(K, N), weight(K, N), None, None, None, None, 1.0)


def test_any_object_with_a_weight_and_adapters_is_a_linear(chain):
    ch = chain.LinearChain([linear(64, 128), linear(128, 64)])
    assert len(ch.layers) == 2
    chain.LinearChain([linear(64, 128), gated(chain, 128, 192), linear(192, 64)], "int8",
                      head=chain.HeadLoss(weight(64, 320)))
    with pytest.raises(ValueError):
        chain.LinearChain([linear(64, 128), linear(64, 128)])
    with pytest.raises(ValueError):
        chain.LinearChain([gated(chain, 64, 128), gated(chain, 64, 128)])
    with pytest.raises(ValueError):
        chain.LinearChain([gated(chain, 64, 128)], head=chain.HeadLoss(weight(64, 320)))
    with pytest.raises(ValueError):
        chain.LinearChain([linear(64, 128)], policy="none")


def test_backward_before_forward(chain):
    with pytest.raises(RuntimeError):
        chain.LinearChain([linear(64, 128)]).backward(None)
    with pytest.raises(RuntimeError):
        chain.LinearChain([]).backward(None)


@pytest.mark.gpu
@pytest.mark.parametrize("policy", ["save", "recompute", "int8"])
def test_a_head_alone(chain, policy):
    """The loss of a head over features that no layer of the chain made."""
    import torch

    import bit_nf4_quantized_pack_b200 as q
    torch.manual_seed(1)
    w = q.quantize(torch.randn(64, 128, device="cuda").to(torch.bfloat16))
    X = torch.randn(9, 64, device="cuda").to(torch.bfloat16)
    y = torch.arange(9, device="cuda")
    y[4] = -100
    head = chain.HeadLoss(w, vocab=100)
    mean, dX, grads = chain.LinearChain([], policy, head=head).loss_backward(X, y)
    want, _, lse = head.forward(X, y)
    assert grads == [] and torch.equal(mean, want) and torch.equal(dX, head.backward(X, lse, y))
