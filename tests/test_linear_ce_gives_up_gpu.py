"""Failure detection in linear cross entropy on the GPU, without a fault: its bounded
waits are given no time, and what it reports is checked."""

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from learned_optimizer_step_gb300 import lm_ops as ops
from tests.gpu_helpers import need_gpu
from tests.test_linear_ce_gpu import check_forward, inputs
from tests.test_train_ops_gpu import gen, guarded

pytestmark = pytest.mark.gpu

GAVE_UP = 2


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


@pytest.mark.parametrize("n,v,d", [(5, 300, 64), (700, 5003, 520)])
def test_waits_that_run_out_are_reported(n, v, d):
    x, w, t, rw = inputs(gen(n), n, v, d, torch.bfloat16)
    need = ops._size_of("lopt_linear_ce_workspace", n, v, d, 1, 0, ops.F32)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    for limit in (10 ** 9, 0, 0, 10 ** 9):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        (loss, a), (lse, b) = guarded((n,), torch.float32), guarded((n,), torch.float32)
        code = ops._load()["lopt_selftest_linear_ce"](
            limit, x.data_ptr(), ops.BF16, n, d, d, w.data_ptr(), v, d, t.data_ptr(), 1, rw.data_ptr(), loss.data_ptr(),
            lse.data_ptr(), work.data_ptr(), need, status.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert code == 0
        torch.cuda.synchronize()
        a(), b()
        if int(status) == GAVE_UP:
            assert limit == 0 and bool(torch.isnan(loss).all()) and bool(torch.isnan(lse).all())
        else:
            assert int(status) == 0 and limit > 0     # a load takes longer than no time
            check_forward((loss, lse), x, w, t, rw)
    check_forward(L.linear_cross_entropy_forward(x, w, t, row_weight=rw), x, w, t, rw)     # the next call is as ever
    L.check_indices()
