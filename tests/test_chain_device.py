"""LinearChain on a device that is not the current one: every call of the layers
and of the head, and the read-back of the status word, run with the tensors'
device current (its launches go to the current device's stream).  The device
and the calls are stand-ins: nothing here needs a GPU."""
import contextlib
from types import SimpleNamespace

import pytest


@pytest.fixture(scope="module")
def chain():
    from tests.conftest import ensure_built
    ensure_built()
    from bit_nf4_quantized_pack_b200 import chain
    return chain


class Tensor:
    """Enough of a CUDA tensor for the chain's own arithmetic."""
    device, is_cuda, dtype = "second", True, None

    def __ne__(self, other):
        return self

    def __truediv__(self, other):
        return self

    def sum(self):
        return self

    def clamp(self, min):
        return self

    def to(self, dtype):
        return self


@pytest.mark.parametrize("policy", ["save", "recompute", "int8"])
@pytest.mark.parametrize("own_status", [True, False])
def test_the_tensors_device_is_current(chain, monkeypatch, policy, own_status):
    current, seen = ["first"], []
    t = Tensor()

    @contextlib.contextmanager
    def on(dev):
        before, current[0] = current[0], dev
        yield
        current[0] = before

    def call(name, result):
        def f(*args, **kw):
            seen.append(name)
            assert current[0] == "second", name
            return result
        monkeypatch.setattr(chain, name, f)
    monkeypatch.setattr(chain._args, "on", on)
    for name, result in (("act8_quantize", t), ("gated_forward", (t, t)), ("linear_forward", (t, t)),
                         ("gated_backward", (t, t, t, t, t)), ("linear_backward", (t, t, t)),
                         ("head_loss_forward", (t, t)), ("head_loss_backward", t), ("new_status", t),
                         ("status_sync", (0, 0))):
        call(name, result)
    w = SimpleNamespace(shape=(64, 64))
    layers = [chain.GatedLayer(w, w, t, t, t, t, 1.0), chain.Layer(w, t, t, 1.0)]
    ch = chain.LinearChain(layers, policy, head=chain.HeadLoss(w))
    status = None if own_status else t
    ch.loss_backward(t, t, status)
    ch.forward(t, status)
    ch.backward(t, status)
    assert current[0] == "first"
    assert {"linear_forward", "linear_backward", "gated_backward", "head_loss_backward"} <= set(seen)
    assert ("status_sync" in seen) == own_status
