"""Block norm on the GPU against float64 (tests/lm_reference.py), at the widths
where the kernels change, with strides, offsets, in-place outputs and rows that are
all zeros."""

import math

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from learned_optimizer_step_gb300 import LoptError
from tests import lm_reference as R
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import DTYPES, gen, guarded, ids, normal, padded

pytestmark = pytest.mark.gpu

# Roundings on the way to a result, in half steps of float32.  A row's sum: at most
# 32 terms one after the other in a thread (128 for rows that are read again, which
# are 512 threads wide), 5 by shuffles, 16 by warps, so 53 (149); half of it through the
# root; some 20 for products, the root and the sigmoid's exponential (2^-22 and the
# rounding of its argument, below 12 here: 17 half steps).
FWD = lambda cols: (32 if cols <= 16384 else 128) + 21 + 40          # noqa: E731
BWD = lambda cols: 3 * FWD(cols)                                     # noqa: E731
EPS = 1e-6


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def inputs(g, rows, cols, dtype, wtype, gate):
    h = normal(g, rows, cols) * torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    return (h.to(dtype), normal(g, rows, cols, dtype=dtype, std=2.0), normal(g, cols, dtype=wtype, mean=1.0, std=0.1),
            normal(g, cols, dtype=wtype, mean=1.0, std=0.1),
            normal(g, rows, cols, dtype=dtype, std=2.0).clamp_(-8, 8) if gate else None)


def check_forward(got, h, r, w1, w2, gate, scale, name=""):
    cols = h.shape[-1]
    (y, x, r1, r2), (sy, sx) = R.norm_forward(h, r, w1, w2, gate, scale, EPS)
    R.within(got[0], y, FWD(cols), sy, name + " y")
    R.within(got[1], x, FWD(cols), sx, name + " summed")
    R.within(got[2], r1, FWD(cols), r1, name + " rstd_post")
    R.within(got[3], r2, 2 * FWD(cols), r2 * (1 + (sx / x.abs().mean(-1, keepdim=True)).amax(-1)), name + " rstd_pre")


def check_backward(got, dy, h, x, r1, r2, w1, w2, gate, scale, ds, name=""):
    rows, cols = h.numel() // h.shape[-1], h.shape[-1]
    want, size = R.norm_backward(dy, h, x, r1, r2, w1, w2, gate, scale, ds)
    for k, what in enumerate(("grad_h", "grad_residual", "grad_gate", "grad_w_post", "grad_w_pre")):
        if want[k] is None:
            assert got[k] is None
            continue
        # A column's sum: the rows of a block one after the other, 24 groups, 8 and 20 partial sums.
        units = BWD(cols) + (math.ceil(rows / 32) + 52 if k > 2 else 0)
        R.within(got[k], want[k], units, size[k], "%s %s" % (name, what))


COLS = [1, 2, 7, 8, 31, 64, 129, 256, 264, 500, 512, 513, 768, 776, 1000, 1024, 1032, 2001, 2048, 2056, 4096, 4104, 5000,
        8192, 8200, 16384, 16400, 20001]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("cols", COLS)
def test_widths(cols, dtype):
    g = gen(cols)
    rows = 3 if cols > 4096 else 11
    gate = cols % 3 != 0
    h, r, w1, w2, gt = inputs(g, rows, cols, dtype, torch.float32 if cols % 2 else dtype, gate)
    got = L.block_norm_forward(h, r, w1, w2, gate=gt, scale=0.7, eps=EPS)
    check_forward(got, h, r, w1, w2, gt, 0.7)
    dy, ds = normal(g, rows, cols, dtype=dtype), normal(g, rows, cols, dtype=dtype) if cols % 5 else None
    x, r1, r2 = got[1:]
    back = L.block_norm_backward(dy, h, x, r1, r2, w1, w2, gate=gt, scale=0.7, grad_summed=ds)
    check_backward(back, dy, h, x, r1, r2, w1, w2, gt, 0.7, ds)


@pytest.mark.parametrize("rows", [0, 1, 2, 455, 3001])
@pytest.mark.parametrize("cols", [96, 768, 2048])
def test_rows(rows, cols):
    g = gen(rows)
    h, r, w1, w2, gt = inputs(g, rows, cols, torch.bfloat16, torch.float32, True)
    got = L.block_norm_forward(h, r, w1, w2, gate=gt, scale=-1.5, eps=EPS)
    dy = normal(g, rows, cols, dtype=torch.bfloat16)
    a, b = torch.full((cols,), 3.0, device="cuda"), torch.full((cols,), 5.0, device="cuda")
    back = L.block_norm_backward(dy, h, *got[1:], w1, w2, gate=gt, scale=-1.5, grad_w_post=a, grad_w_pre=b)
    if rows == 0:
        assert not bool(a.any()) and not bool(b.any())
        return
    check_forward(got, h, r, w1, w2, gt, -1.5)
    check_backward(back, dy, h, *got[1:], w1, w2, gt, -1.5, None)
    first = a.clone(), b.clone()
    L.block_norm_backward(dy, h, *got[1:], w1, w2, gate=gt, scale=-1.5, grad_w_post=a, grad_w_pre=b, accumulate=True)
    assert torch.equal(a, 2 * first[0]) and torch.equal(b, 2 * first[1])


@pytest.mark.parametrize("cols,extra,shift", [(768, 8, 8), (768, 3, 1), (101, 5, 0), (2048, 0, 4), (20000, 7, 2)])
def test_strides_offsets_and_guards(cols, extra, shift):
    g = gen(cols + extra)
    rows, dtype = 9, torch.float16
    h, r, w1, w2, gt = inputs(g, rows, cols, dtype, torch.float32, True)
    want = L.block_norm_forward(h, r, w1, w2, gate=gt, scale=0.5)
    ph, pr, pg = (padded(t, extra, shift)[0] for t in (h, r, gt))
    (y, ya), (s, sa) = guarded((rows, cols), dtype, shift), guarded((rows, cols), dtype, shift)
    (r1, ra), (r2, rb) = guarded((rows,), torch.float32), guarded((rows,), torch.float32)
    got = L.block_norm_forward(ph, pr, w1, w2, gate=pg, scale=0.5, out=y, summed=s, rstd_post=r1, rstd_pre=r2)
    for a, b in zip(got, want):     # another kernel adds in another order
        assert float((a.double() - b.double()).norm()) <= 4e-3 * float(b.double().norm())
    check_forward(got, h, r, w1, w2, gt, 0.5)
    dy = padded(normal(g, rows, cols, dtype=dtype), extra, shift)[0]
    outs = [guarded((rows, cols), dtype, shift) for _ in range(3)] + [guarded((cols,), torch.float32) for _ in range(2)]
    back = L.block_norm_backward(dy, ph, s, r1, r2, w1, w2, gate=pg, scale=0.5, grad_h=outs[0][0], grad_residual=outs[1][0],
                                 grad_gate=outs[2][0], grad_w_post=outs[3][0], grad_w_pre=outs[4][0])
    check_backward(back, dy, h, s, r1, r2, w1, w2, gt, 0.5, None)
    for whole in [ya, sa, ra, rb] + [o[1] for o in outs]:
        whole()


@pytest.mark.parametrize("cols", [256, 2048, 20000])
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_in_place(cols, dtype):
    g = gen(4)
    h, r, w1, w2, gt = inputs(g, 300 if cols < 4096 else 5, cols, dtype, torch.float32, True)
    want = L.block_norm_forward(h, r, w1, w2, gate=gt)
    h2, r2 = h.clone(), r.clone()
    got = L.block_norm_forward(h2, r2, w1, w2, gate=gt, out=h2, summed=r2)
    assert got[0] is h2 and all(map(torch.equal, got, want))
    dy, ds = torch.randn_like(h), torch.randn_like(h)
    x, a, b = want[1:]
    back = L.block_norm_backward(dy, h, x, a, b, w1, w2, gate=gt, grad_summed=ds)
    c = [t.clone() for t in (dy, h, x, gt, ds)]
    again = L.block_norm_backward(c[0], c[1], c[2], a, b, w1, w2, gate=c[3], grad_summed=c[4], grad_h=c[0],
                                  grad_residual=c[4], grad_gate=c[3])
    assert all(map(torch.equal, again, back))


def test_rows_of_zeros_and_special_values():
    cols = 512
    g = gen(2)
    h, r, w1, w2, gt = inputs(g, 6, cols, torch.float32, torch.float32, True)
    h[0] = 0
    r[0] = 0                      # summed is then 0 too: rstd = eps^-1/2, y = 0
    gt[1, ::2], gt[1, 1::2] = math.inf, -math.inf
    gt[2, :2] = torch.tensor([200.0, -200.0])
    h[3, 5] = math.nan
    y, x, r1, r2 = L.block_norm_forward(h, r, w1, w2, gate=gt)
    assert not bool(y[0].any()) and float(r2[0]) == pytest.approx(EPS ** -0.5, rel=1e-6)
    assert torch.equal(x[1, 1::2], r[1, 1::2]) and bool(torch.isfinite(y[[0, 1, 2, 4, 5]]).all())
    assert bool(torch.isnan(y[3]).all())
    dy = torch.ones_like(h)
    dh, dx, dg, d1, d2 = L.block_norm_backward(dy, h, x, r1, r2, w1, w2, gate=gt)
    assert not bool(dg[1].any()) and bool(torch.isfinite(dh[[0, 1, 2, 4, 5]]).all())
    assert bool(torch.isnan(dh[3]).all())


def test_gradients_against_differences():
    """In float64 the formulas of the reference are the derivative of its forward pass."""
    g = torch.Generator()
    g.manual_seed(1)
    t = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)   # noqa: E731
    h, r, w1, w2, gt, dy, ds = t(4, 13), t(4, 13), t(13), t(13), t(4, 13), t(4, 13), t(4, 13)

    def value(*a):
        (y, x, _, _), _ = R.norm_forward(a[0], a[1], a[2], a[3], a[4], 0.7, EPS)
        return (y * dy).sum() + (x * ds).sum()

    args = [h, r, w1, w2, gt]
    (_, x, r1, r2), _ = R.norm_forward(h, r, w1, w2, gt, 0.7, EPS)
    dh, dx, dg, d1, d2 = R.norm_backward(dy, h, x, r1, r2, w1, w2, gt, 0.7, ds)[0]
    for k, d in ((0, dh), (1, dx), (2, d1), (3, d2), (4, dg)):
        v = torch.randn(args[k].shape, generator=g, dtype=torch.float64)
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + 1e-6 * v, args[k] - 1e-6 * v
        slope = (value(*up) - value(*down)) / 2e-6
        assert abs(float(slope - (d * v).sum())) <= 1e-6 * float((d * v).abs().sum()), k


def test_refusals():
    g = gen(1)
    h, r, w1, w2, gt = inputs(g, 4, 64, torch.bfloat16, torch.float32, True)
    y, x, r1, r2 = L.block_norm_forward(h, r, w1, w2, gate=gt)
    for call, error in ((lambda: L.block_norm_forward(h, r[:3], w1, w2), ValueError),
                        (lambda: L.block_norm_forward(h, r.float(), w1, w2), ValueError),
                        (lambda: L.block_norm_forward(h, r, w1.half(), w2.half()), TypeError),
                        (lambda: L.block_norm_forward(h, r, w1, w2.bfloat16()), TypeError),
                        (lambda: L.block_norm_forward(h, r, w1[:32], w2[:32]), ValueError),
                        (lambda: L.block_norm_forward(h, r.cpu(), w1, w2), TypeError),
                        (lambda: L.block_norm_forward(h, r, w1, w2, eps=-1.0), LoptError),
                        (lambda: L.block_norm_forward(h, r, w1, w2, scale=math.inf), LoptError),
                        (lambda: L.block_norm_forward(h, r, w1, w2, out=x, summed=x), LoptError),
                        (lambda: L.block_norm_forward(h.t(), r.t(), w1, w2), ValueError),
                        (lambda: L.block_norm_backward(y, h, x, r1[:2], r2, w1, w2), ValueError),
                        (lambda: L.block_norm_backward(y, h, x, r1, r2, w1, w2, grad_gate=y), ValueError),
                        (lambda: L.block_norm_backward(y, h, x, r1, r2, w1, w2, accumulate=True), ValueError)):
        with pytest.raises(error):
            call()
