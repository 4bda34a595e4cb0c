"""Distillation over the accepted range of temperatures on the GPU, and its
ends, in every kernel."""

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from learned_optimizer_step_gb300 import LoptError
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import DTYPES, check_distill, distill_inputs, gen, ids, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


@pytest.mark.parametrize("T", [1e-30, 1e-25, 1e-22, 1e-19, 1e-10, 1e-3, 30.0, 300.0, 1e3])
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_temperatures(dtype, T):
    for rows, cols, top in ((5, 64, 64), (4, 1000, 20), (3, 3001, 60), (3, 50257, 64), (2, 500009, 9)):
        g = gen(rows + cols)
        z, t, i = distill_inputs(g, rows, cols, top, dtype, torch.float32, torch.int64)
        if top == cols:
            # every class, once: the loss does not grow with T
            t, i = normal(g, rows, cols), torch.argsort(torch.rand(rows, cols, generator=g, device="cuda"), 1)
        w = torch.rand(rows, generator=g, device="cuda") + 0.5
        loss, grad = L.distill_forward_backward(z, t, i, T, row_weight=w)
        check_distill(z, t, i, float(torch.tensor(T)), w, loss, grad, "%d classes" % cols)
        assert torch.equal(loss, L.distill_forward(z, t, i, T, row_weight=w))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=ids)
def test_a_wanted_class_at_the_lowest_value(dtype):
    """Its loss is T times the distance: in range for a small T."""
    g = gen(8)
    for cols in (64, 3001, 50257, 950003):
        z = normal(g, 3, cols, dtype=dtype)
        z[:, 5] = torch.finfo(dtype).min
        i = torch.tensor([[5, 1], [5, 5], [2, 5]], device="cuda")
        t = torch.zeros(3, 2, device="cuda")
        for T in (1e-3, 2.0 ** -5):
            loss, grad = L.distill_forward_backward(z, t, i, T)
            check_distill(z, t, i, float(torch.tensor(T)), None, loss, grad, "%d classes, T=%g" % (cols, T))


def test_a_sum_of_probabilities_that_rounds_up_does_not_overflow():
    """Float32 slots all at the lowest value: their p add up to 1 and a bit in
    some rows, the loss is half or a quarter of the largest number."""
    g = gen(9)
    low = torch.finfo(torch.float32).min
    for cols in (64, 3001, 50257, 500009):
        rows = 300 if cols < 4000 else 40
        z = normal(g, rows, cols)
        z[:, :40] = low
        for top in (5, 23, 40):
            i = torch.argsort(torch.rand(rows, 40, generator=g, device="cuda"), 1)[:, :top].contiguous()
            t = normal(g, rows, top)
            for T in (0.5, 0.25):
                loss, grad = L.distill_forward_backward(z, t, i, T)
                assert torch.isfinite(loss).all(), (cols, top, T)
                check_distill(z, t, i, T, None, loss, grad, "%d classes, T=%g" % (cols, T))
                assert torch.equal(loss, L.distill_forward(z, t, i, T))


def test_temperatures_beyond_are_refused():
    z, t = torch.zeros(2, 8, device="cuda"), torch.zeros(2, 1, device="cuda")
    i = torch.zeros(2, 1, dtype=torch.int64, device="cuda")
    for T in (1e-31, 1001.0, 1e5, 1e19, 1e30, -2.0):
        with pytest.raises(LoptError) as e:
            L.distill_forward(z, t, i, T)
        assert e.value.code == -1, T
