"""MoEBlock runs on its input's device and not on the current one (CPU only:
the device switch and the operators are stood in for)."""
import pytest

from sparse_mixture_experts_noisy_b200 import moe


class Device:
    """Stands in for the switch to the tensors' device."""

    def __init__(self):
        self.inside = False

    def __enter__(self):
        self.inside = True

    def __exit__(self, *a):
        self.inside = False


@pytest.fixture
def device(monkeypatch):
    at, seen = Device(), []
    monkeypatch.setattr(moe, "_elsewhere", lambda x, stream: None if at.inside else at)
    monkeypatch.setattr(moe, "_cuda", lambda t, name: None)

    def note(name, result):
        def f(*a, **k):
            seen.append((name, at.inside))
            return result
        return f

    class Grads(dict):
        def add_(self, other):
            return self

    tensor = Grads()
    monkeypatch.setattr(moe, "moe_layer_norm", note("norm", (tensor, tensor, tensor, tensor)))
    monkeypatch.setattr(moe, "moe_linear", lambda *a, **k: note("linear", (tensor, tensor) if k.get("keep_z") else tensor)())
    monkeypatch.setattr(moe, "moe_route", note("route", (tensor, tensor, None)))
    d = dict(x_gathered=tensor, offsets=tensor, counts=tensor, slot=tensor)
    monkeypatch.setattr(moe, "moe_dispatch", note("dispatch", d))
    monkeypatch.setattr(moe, "moe_expert_ffn_train", note("ffn", (tensor, tensor)))
    monkeypatch.setattr(moe, "moe_combine", note("combine", tensor))
    monkeypatch.setattr(moe, "moe_backward", lambda *a, **k: note("backward", dict(dx=tensor, ws=None))())
    monkeypatch.setattr(moe, "moe_linear_backward", note("linear_backward", dict(dx=tensor, dW=tensor, db=tensor)))
    monkeypatch.setattr(moe, "moe_layer_norm_backward", note("norm_backward", dict(dx=tensor)))

    class Layer:
        act, b_up, b_down, b_g = moe.ACT_RELU, None, None, None
        W_g = W_up = W_down = tensor
        E, k, cf, sigma = 4, 2, None, 0.0

        def __call__(self, n, noise=None):
            return note("layer", tensor)()

    return seen, moe.MoEBlock(Layer(), shared=(tensor, None, tensor, None)), tensor, at


def test_every_operator_runs_on_the_inputs_device(device):
    seen, block, x, at = device
    block(x)
    saved = block.train(x)[2]
    block.backward(x, x, saved)
    names = {n for n, _ in seen}
    assert names == {"norm", "linear", "layer", "route", "dispatch", "ffn", "combine", "backward", "linear_backward",
                     "norm_backward"}
    assert all(inside for _, inside in seen), [n for n, inside in seen if not inside]
    assert not at.inside
