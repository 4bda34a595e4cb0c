"""How exact linear cross entropy's gradients are on the GPU, beside float64: what the
parts of G and the length of the tensor cores' sums leave."""

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from tests import lm_reference as R
from tests.gpu_helpers import need_gpu
from tests.test_linear_ce_gpu import HALF, inputs
from tests.test_train_ops_gpu import gen, ids, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("n", [200, 700])
@pytest.mark.parametrize("extra", [24, 5])
def test_a_block_of_columns_has_the_bits_of_a_buffer_of_its_own(n, extra, dtype):
    """A 32-bit grad_weight inside a wider buffer, on 16-byte rows and off them."""
    v, d = 900, 72
    x, w, t, rw = inputs(gen(n), n, v, d, dtype)
    _, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    wide = torch.full((v, d + extra), 5.0, device="cuda")
    part = wide[:, extra // 3:extra // 3 + d]
    for accumulate in (False, True):
        want, got = torch.full((v, d), 0.25, device="cuda"), part.fill_(0.25)
        L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, grad_weight=want, accumulate=accumulate)
        L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, grad_weight=got, accumulate=accumulate)
        assert torch.equal(got, want)
    part.fill_(5.0)
    assert bool((wide == 5).all())


def test_without_grad_weight_over_several_chunks():
    """A frozen table: its gradient is not asked for.  G of 4,099 tokens, 50,257 classes is
    two chunks.  grad_x is the same to what one part of G leaves, half a step of an entry."""
    x, w, t, rw = inputs(gen(3), 4099, 50257, 128, torch.bfloat16)
    _, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    dx, none = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, need_weight=False)
    want, _, g = R.ce_backward(x, w, t, lse, rw)
    assert none is None
    size = g.abs() @ w.double().abs()
    R.within(dx, want, 1, size * (2.0 ** -8 / R.U), "grad_x")
