"""The example model end to end: the operators together, as a layer's forward,
its single-token form and its training step use them."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.small_route]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("ternary_mixer", os.path.join(ROOT, "examples", "ternary_mixer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("width,length", [(512, 300), (243, 40)])
def test_prefill_tokens_and_training(example, width, length):
    off, losses, state = example.main(width=width, batch=2, length=length, steps=12)
    # the recurrence's float sums differ between the two orders, which may move a
    # code of the second norm by one step (1/127 of the row's largest value) here
    # and there; a row sums width / 3 * 2 such terms at most, most of them unmoved
    assert off < 0.1
    assert state < 1e-3
    assert losses[-1] < losses[0]


def test_gradients_by_differences_of_the_norm_gain(example):
    """The straight-through gradient of gamma_out points downhill: a step along
    it lowers a loss that goes through the quantizer and the ternary product."""
    m = example.TernaryMixer(256, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn((2, 64, 256), generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn((2, 64, 256), generator=g, device="cuda")
    saved = {}
    y, _ = m.forward(x, saved=saved)
    dy = (y.float() - target).to(torch.bfloat16)
    _, grads = m.backward(dy, saved)
    before = (y.float() - target).square().sum()
    for param, grad in grads:
        if param is m.gamma_out or param is m.out.bias:
            keep = param.clone()
            param -= 0.05 * grad / grad.norm()
            after = (m.forward(x)[0].float() - target).square().sum()
            param.copy_(keep)
            assert after < before
