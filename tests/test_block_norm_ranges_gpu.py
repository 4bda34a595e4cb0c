"""Block norm on the GPU on rows of very large and very small size: what the formulas give
is in range, and so is what the kernels make on the way."""

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from tests import lm_reference as R
from tests.gpu_helpers import need_gpu
from tests.test_block_norm_gpu import FWD, check_backward, inputs
from tests.test_train_ops_gpu import gen, ids, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=ids)
@pytest.mark.parametrize("cols", [96, 500, 768, 2048, 8200])
@pytest.mark.parametrize("of_h,of_residual", [(1e14, 1e14), (1e14, 1.0), (1.0, 1e14), (1e17, 1e17), (1e17, 1.0), (1.0, 1e17),
                                              (1e-16, 1e-16), (1e-16, 1.0), (1.0, 1e-16), (1e17, 1e-16), (1e-16, 1e17)])
def test_gradients_of_rows_of_any_size(of_h, of_residual, cols, dtype):
    g = gen(cols)
    h, r, w1, w2, gate = inputs(g, 9, cols, torch.float32, torch.float32, cols != 768)
    h, r = (h * of_h).to(dtype), (r * of_residual).to(dtype)
    gate = None if gate is None else gate.to(dtype)
    scale = 0.7 * min(of_residual, 1.0)       # summed is of residual's size, or of 1
    y, x, r1, r2 = L.block_norm_forward(h, r, w1, w2, gate=gate, scale=scale, eps=0.0)
    # summed is rounded once more than what its root is of.
    for got, rows, more in ((r1, h, 0.0), (r2, x, R.half_step(dtype))):
        want = rows.double().square().mean(-1).rsqrt()
        assert float(((got.double() - want) / want).abs().max()) <= FWD(cols) * R.U + more
    dy, ds = normal(g, 9, cols, dtype=dtype), (normal(g, 9, cols) / max(of_residual, 1.0)).to(dtype)
    for past in (None, ds):
        back = L.block_norm_backward(dy, h, x, r1, r2, w1, w2, gate=gate, scale=scale, grad_summed=past)
        check_backward(back, dy, h, x, r1, r2, w1, w2, gate, scale, past, "%g %g" % (of_h, of_residual))
