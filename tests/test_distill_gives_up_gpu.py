"""Failure detection in the distillation kernel on the GPU, without a fault:
its bounded waits are given no time at all, and what it reports is checked."""

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from learned_optimizer_step_gb300 import train_ops as ops
from tests import train_reference as R
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import check_distill, distill_inputs, gen, guarded

pytestmark = pytest.mark.gpu

GAVE_UP = 2


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def selftest(limit, z, t, i, w, loss, grad, status):
    code = ops._load()["lopt_selftest_distill"](
        limit, z.data_ptr(), ops._TYPES[z.dtype], *z.shape, z.stride(0), t.data_ptr(), ops.F32, t.stride(0), i.data_ptr(),
        ops.I64, i.stride(0), t.shape[1], 1.5, w.data_ptr(), loss.data_ptr(), 0 if grad is None else grad.data_ptr(),
        z.shape[1], status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert code == 0
    torch.cuda.synchronize()


# One, two and eight persistent blocks to a row, with several rows to each.
@pytest.mark.parametrize("dtype,rows,cols,top", [(torch.bfloat16, 2500, 9001, 40), (torch.bfloat16, 2000, 50257, 64),
                                                 (torch.float32, 300, 131075, 200)])
def test_waits_that_run_out_are_reported(dtype, rows, cols, top):
    g = gen(rows + cols)
    z, t, i = distill_inputs(g, rows, cols, top, dtype, torch.float32, torch.int64)
    w = torch.rand(rows, generator=g, device="cuda") + 0.5
    w[torch.rand(rows, generator=g, device="cuda") < 0.2] = 0.0
    want, want_grad = R.distill(z, t, i, 1.5, w)
    b_loss, b_grad = R.distill_bounds(z, t, i, 1.5, want_grad, w)
    b_grad += R.rounded(want_grad, dtype) * 1.01
    for limit, with_grad in ((10 ** 9, True), (0, True), (0, False), (2000, True), (2000, False)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        loss, whole_l = guarded((rows,), torch.float32)
        grad, whole_g = guarded((rows, cols), dtype)
        selftest(limit, z, t, i, w, loss, grad if with_grad else None, status)
        whole_l(), whole_g()
        lost = torch.isnan(loss)
        print("limit %d ns, gradient %s: %d of %d rows lost" % (limit, with_grad, int(lost.sum()), rows))
        assert int(status) == (GAVE_UP if lost.any() else 0)
        assert limit < 10 ** 9 or not lost.any()
        fine = ~lost
        R.check(loss[fine], want[fine], b_loss[fine], "loss")
        if with_grad:
            R.check(grad[fine], want_grad[fine], b_grad[fine], "grad")
    loss, grad = L.distill_forward_backward(z, t, i, 1.5, row_weight=w)     # the next call is as ever
    check_distill(z, t, i, 1.5, w, loss, grad, "after")
    L.check_indices()


def test_limits_are_checked():
    one = torch.zeros(1, 8, device="cuda")
    i = torch.zeros(1, 1, dtype=torch.int64, device="cuda")
    out = torch.zeros(1, device="cuda")
    for limit in (-1, 10 ** 9 + 1):
        assert ops._load()["lopt_selftest_distill"](limit, one.data_ptr(), 0, 1, 8, 8, one.data_ptr(), 0, 1, i.data_ptr(), 1, 1,
                                                    1, 1.0, 0, out.data_ptr(), 0, 0, 0, 0) == -1
