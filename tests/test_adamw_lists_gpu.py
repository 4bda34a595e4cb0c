"""AdamW on the GPU over lists longer than its launches, and without elements."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from tests.gpu_helpers import need_gpu
from tests.test_adamw_gpu import H, check, make, opt

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


@pytest.mark.parametrize("count", [6400, 6401, 13007])
def test_clipping_of_more_tensors_than_partial_sums_hold(count):
    """400 tensors a launch of the norm, 16 launches with partial sums of their own."""
    rng = np.random.default_rng(count)
    sizes = rng.integers(1, 40, count)
    sizes[::997] = 5000                     # launches of more blocks, early and late
    ts = [make(rng, int(n), False) for n in sizes]
    norm = opt([t for t, _ in ts]).step(2, H["lr"], max_norm=0.5)
    want = math.sqrt(math.fsum(float(x) ** 2 for _, o in ts for x in o["g"]))
    assert abs(float(norm) - want) <= want * 2.0 ** -24 * 1.0001
    clip = np.float32(min(1.0, 0.5 / (want + 1e-6)))
    for k in list(range(0, count, 83)) + [count - 1]:
        check(*ts[k], k, 2, 2, clip)


def test_the_norm_of_no_elements_is_written_in_order():
    """Its kernel may be set up while the one before still runs, which writes the same word:
    the norm's place is an element of a gradient, which comes first."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, w = (torch.randn(n, 256, generator=g, device="cuda").to(torch.bfloat16) for n in (8192, 20000))
    t = torch.zeros(8192, dtype=torch.int64, device="cuda")
    _, lse = L.linear_cross_entropy_forward(x, w, t)
    grad = torch.empty(20000, 256, device="cuda")
    empty = lambda: torch.zeros(0, device="cuda")   # noqa: E731
    a = L.AdamW([L.AdamWTensor(empty(), empty(), empty(), empty())])
    for place in (grad[19999, 255], grad[0, 0]):
        for _ in range(5):
            L.linear_cross_entropy_backward(x, w, t, lse, grad_weight=grad, need_x=False)
            norm = a.step(1, 0.1, max_norm=1.0, norm=place)
            assert float(norm) == 0.0
