"""More sizes for the training operators' kernels on the GPU: the ranges at
whose ends another kernel, another block size or a fallback inside a kernel
takes over, and batches that give every block several rows."""

import math

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from tests import train_reference as R
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import (DTYPES, check_distill, distill_inputs, gen, guarded, ids, norm_inputs, normal,
                                      token_lists)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


# Lists of one id that no block can keep in shared memory; tables whose ids
# need 32 warps to a block and more than 128 blocks; positions that do not fit
# an entry of the sort.
@pytest.mark.parametrize("n,rows,cols", [(150000, 257, 8), (150001, 70001, 3), (3000, 66000, 4), (2500, 300001, 2),
                                         (16383, 1000, 16), (16384, 1000, 16), (4300000, 3, 1)])
def test_embedding_backward_ranges(n, rows, cols):
    g = gen(n + rows)
    for k, (kind, index) in enumerate(token_lists(g, n, rows)):
        dy = normal(g, n, cols, dtype=DTYPES[k % 3])
        index = index.to(torch.int64 if k % 2 else torch.int32)
        want, bound = R.embed_backward(dy, index, rows, 0.75)
        out, whole = guarded((rows, cols), torch.float32)
        L.embedding_backward(dy, index, rows, 0.75, out=out)
        R.check(out, want, bound, kind)
        whole()
        assert torch.equal(out, L.embedding_backward(dy, index, rows, 0.75)), kind


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(1300, 64), (901, 256), (640, 1024), (500, 2048), (330, 4096), (321, 5001),
                                       (310, 8200), (305, 2050), (40, 17000), (160, 1032), (310, 2056), (170, 6000), (1001, 16)])
def test_layernorm_many_rows(dtype, rows, cols):
    g = gen(rows * 7 + cols)
    x, w, b = norm_inputs(g, rows, cols, dtype, torch.float32)
    res, dy = normal(g, rows, cols, dtype=dtype), normal(g, rows, cols, dtype=dtype)
    y, sm, mean, rstd = R.norm_forward(x, w, b, 1e-5, res)
    by, _, bm, br = R.norm_forward_bounds(sm, mean, rstd, y, w, b, dtype)
    got = L.layernorm_forward(x, w, b, residual=res)
    R.check(got[0], y, by, "y")
    R.check(got[2], mean, bm, "mean")
    R.check(got[3], rstd, br, "rstd")
    s, mean, rstd = got[1], got[2], got[3]
    dx, dw, db = R.norm_backward(dy, s, mean, rstd, w, res)
    bx, bw, bb = R.norm_backward_bounds(dy, s, mean, rstd, w, dx, dtype, res)
    back = L.layernorm_backward(dy, s, mean, rstd, w, grad_residual=res)
    for a, want, bound, what in zip(back, (dx, dw, db), (bx, bw, bb), ("dx", "dweight", "dbias")):
        R.check(a, want, bound, what)
    again = L.layernorm_backward(dy, s, mean, rstd, w, grad_residual=res)
    assert all(torch.equal(a, c) for a, c in zip(back, again))


# Short rows with lists in a lane each, in shared memory, and just too long for
# that; rows for clusters of one, two and eight blocks, several to a cluster.
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("rows,cols,top", [(301, 500, 32), (301, 500, 33), (300, 700, 200), (203, 1000, 256),
                                           (203, 1000, 257), (2000, 2500, 8), (1500, 5003, 40), (1300, 9001, 129),
                                           (700, 32003, 64), (400, 100003, 5)])
def test_distill_many_rows(dtype, rows, cols, top):
    g = gen(rows + 3 * cols + top)
    z, t, i = distill_inputs(g, rows, cols, top, dtype, torch.float32, torch.int64)
    i[::3, top // 2:] = i[::3, :top - top // 2]          # classes listed twice
    i[5::11] = -1                                        # rows without a list
    w = torch.rand(rows, generator=g, device="cuda") + 0.5
    w[torch.rand(rows, generator=g, device="cuda") < 0.3] = 0.0
    w[rows // 2:rows // 2 + 40] = 0.0                    # a run that is not counted
    grad, whole = guarded((rows, cols), dtype)
    loss, _ = L.distill_forward_backward(z, t, i, 1.7, row_weight=w, grad=grad)
    whole()
    check_distill(z, t, i, 1.7, w, loss, grad, "weights")
    assert torch.equal(loss, L.distill_forward(z, t, i, 1.7, row_weight=w))
    assert not grad[w == 0].any() and not grad[5::11].any()
    L.check_indices()


def test_offsets_beyond_32_bits():
    """A table and logits whose elements number more than 2^32: the last rows."""
    rows, cols = 70000, 65536                             # 4.6e9 elements of two bytes
    table = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = gen(2)
    table[-2:] = normal(g, 2, cols, dtype=torch.bfloat16)
    index = torch.tensor([rows - 1, 0, rows - 2], device="cuda")
    out = L.embedding_forward(table, index)
    assert torch.equal(out, table[index])
    x, w = table[-2:], torch.ones(cols, device="cuda")
    y, mean, rstd = L.layernorm_forward(table, w)
    want = L.layernorm_forward(x.clone(), w)
    assert torch.equal(y[-2:], want[0]) and torch.equal(mean[-2:], want[1]) and not y[-3].any()
    del y
    t = torch.zeros(rows, 2, device="cuda")
    i = torch.tensor([[7, 9]], device="cuda").expand(rows, 2)
    weight = torch.zeros(rows, device="cuda")
    weight[-3:] = 1.0
    loss = L.distill_forward(table, t, i, row_weight=weight)
    assert torch.equal(loss[-2:], L.distill_forward(x.clone(), t[-2:], i[-2:])) and not loss[:-3].any()
    assert abs(float(loss[-3]) - (math.log(cols) - math.log(2))) < 1e-5


def test_workspaces_after_release():
    g = gen(8)
    dy = normal(g, 300, 64)
    index = torch.randint(0, 90, (300,), generator=g, device="cuda")
    a = L.embedding_backward(dy, index, 90)
    L.release_workspaces()
    assert torch.equal(a, L.embedding_backward(dy, index, 90))
    small = L.embedding_backward(dy[:5], index[:5], 90)      # a workspace larger than it needs
    big = L.embedding_backward(dy.repeat(40, 1), index.repeat(40), 90)
    R.check(small, *R.embed_backward(dy[:5], index[:5], 90, 1.0), "small")
    R.check(big, *R.embed_backward(dy.repeat(40, 1), index.repeat(40), 90, 1.0), "big")
