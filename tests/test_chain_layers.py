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
