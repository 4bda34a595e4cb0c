"""The example that runs the training operators together with the learned
optimizer's step: its gradients against autograd in float64, and its loss
over a few steps."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_small_lm.py")


@pytest.fixture(scope="module")
def example():
    need_gpu()
    spec = importlib.util.spec_from_file_location("distill_small_lm", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_are_those_of_autograd(example):
    """Activations are bfloat16 (a rounding of 2^-9 of their size each): the
    gradients agree with float64 autograd to a few of those in norm."""
    model, teacher = example.Model(3), example.Teacher(4)
    tokens, top, index = teacher.batch(512)
    loss = model.loss_and_gradients(tokens, top, index)
    p = {k: v.double().requires_grad_() for k, v in model.params.items()}
    W = example.WIDTH

    def norm(x, w, b):
        m = x.mean(1, keepdim=True)
        v = ((x - m) ** 2).mean(1, keepdim=True)
        return (x - m) / torch.sqrt(v + 1e-5) * w + b
    x = p["table"][tokens] * W ** 0.5
    s = norm(x, p["n1.w"], p["n1.b"]) @ p["w1"] + x
    logq = torch.log_softmax(norm(s, p["n2.w"], p["n2.b"]) @ p["head"], 1)
    logp = torch.log_softmax(top.double(), 1)
    want = (logp.exp() * (logp - logq.gather(1, index))).sum(1)
    want.mean().backward()
    want = want.detach()
    assert float((loss.double() - want).abs().max()) < 0.02 * float(want.abs().max())
    for k in p:
        off = float((model.grads[k].double() - p[k].grad).norm() / p[k].grad.norm())
        assert off < 16 * 2.0 ** -9, (k, off)


def test_the_loss_falls(example):
    losses = example.main(60, show=False)
    assert losses[-1] < 0.7 * losses[0], losses[::10]
