"""Linear cross entropy on the GPU against float64 (tests/lm_reference.py): sizes on
and beside the tiles' edges, masks, strides, chunks of the vocabulary, gradients in
16 and in 32 bits."""

import math

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from learned_optimizer_step_gb300 import LoptError
from tests import lm_reference as R
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import gen, guarded, ids, normal, padded

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def inputs(g, n, v, d, dtype, padding=0.2, weights=True, index=torch.int64):
    w = normal(g, v, d, dtype=dtype, std=d ** -0.5)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    known = torch.rand(n, 1, generator=g, device="cuda") * 12
    x = (normal(g, n, d) + known * w[t].float()).to(dtype)
    t[torch.rand(n, generator=g, device="cuda") < padding] = -1
    rw = torch.rand(n, generator=g, device="cuda") if weights else None
    return x, w, t.to(index), rw


def cut(steps):
    """Half steps of float32 that `steps` steps of K = 16 on the tensor cores may cut
    from a sum, four each: their products are aligned to the largest term and cut
    within its last bits."""
    return 4 * steps


def logit_units(d):
    # Segments of 2048 of K, their sums added with a rounding each.
    return cut(math.ceil(min(d, 2048) / 16)) + math.ceil(d / 2048) + 4


def check_forward(got, x, w, t, rw):
    loss, lse, size = R.ce_forward(x, w, t, rw)
    # Off by the logits' errors; the sum of V exponentials (128 in a row, then by tiles:
    # 128 + 64), each 2^-22 off and its argument rounded (|z - max| < 64: 100 half
    # steps), the logarithm's last bits.
    units = logit_units(x.shape[-1])
    R.within(got[1], lse, 1, units * size + 300 + 4 * lse.abs(), "lse")
    weight = 1.0 if rw is None else rw.double()
    R.within(got[0], loss, 1, weight * (2 * units * size + 300 + 8 * lse.abs()) + 4 * loss, "loss")


def check_backward(dx, dw, x, w, t, lse, rw):
    n, d, v = x.shape[0], x.shape[1], w.shape[0]
    rx, rd, g = R.ce_backward(x, w, t, lse, rw)
    _, _, size = R.ce_forward(x, w, t, rw)
    live = g.abs().sum(1) > 0
    xs = torch.where(live[:, None], x.double(), 0.0).abs()
    weight = (torch.ones(n, dtype=torch.float64, device="cuda") if rw is None else rw.double()) * live
    # An entry of G: e^z is off by z's error, 2^-22 and its argument's rounding.
    p = torch.exp(x.double() @ w.double().t() - lse.double()[:, None]) * weight[:, None]
    soft = p * (logit_units(d) * size + 200)[:, None]
    hit = torch.zeros_like(p)
    hit[torch.arange(n, device="cuda"), t.long().clamp(0, v - 1)] = weight * (4 * d ** 0.5 * size + 200)
    entry = (soft + hit) * R.U
    top = float(weight.max())
    one = R.half_step(x.dtype)
    # Rounded to 16 bits, at 2^15 / the largest weight; fp16's smallest step is 2^-24.
    floor = top * 2.0 ** -15 * 2.0 ** -25 if x.dtype is torch.float16 else 0.0
    if dx is not None:
        e = entry + one * g.abs() + floor
        R.within(dx, rx, 1, (e @ w.double().abs() + R.U * (cut(v / 16) + 70) * (g.abs() @ w.double().abs())) / R.U, "grad_x")
    if dw is not None:
        fp32 = dw.dtype is torch.float32
        e = entry + (one * one * 1.01 if fp32 else one) * g.abs() + floor
        sums = cut(2 * n / 16) + n + 80       # the targets' rows: one after the other
        R.within(dw, rd, 1, (e.t() @ xs + R.U * sums * (g.abs().t() @ xs)) / R.U, "grad_weight")


CASES = [(1, 1, 1), (1, 2, 8), (2, 255, 64), (3, 256, 65), (7, 257, 63), (128, 300, 128), (129, 511, 72), (255, 512, 200),
         (256, 1000, 256), (257, 1025, 264), (300, 5003, 101), (511, 129, 768), (513, 2049, 96), (1030, 777, 520)]


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("n,v,d", CASES)
def test_sizes(n, v, d, dtype):
    g = gen(n + v)
    x, w, t, rw = inputs(g, n, v, d, dtype, weights=n % 2 == 0, index=torch.int32 if v % 2 else torch.int64)
    loss, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    check_forward((loss, lse), x, w, t, rw)
    for kind in (torch.float32, dtype):
        gw = torch.full((v, d), math.nan, dtype=kind, device="cuda")
        dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, grad_weight=gw)
        check_backward(dx, dw, x, w, t, lse, rw)
    L.check_indices()


@pytest.mark.parametrize("dtype", HALF, ids=ids)
def test_wide_and_long(dtype):
    for n, v, d in ((130, 700, 4100), (20, 40000, 72), (3000, 400, 64)):
        x, w, t, rw = inputs(gen(d), n, v, d, dtype)
        loss, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
        check_forward((loss, lse), x, w, t, rw)
        dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw)
        check_backward(dx, dw, x, w, t, lse, rw)


def test_several_chunks_of_the_vocabulary():
    """G of 40,000 tokens in two parts is 160 KB per class: chunks of 1,536 classes."""
    n, v, d = 40000, 5000, 40
    x, w, t, rw = inputs(gen(3), n, v, d, torch.bfloat16)
    loss, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    check_forward((loss, lse), x, w, t, rw)
    for kind in (torch.float32, torch.bfloat16):
        dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw,
                                                 grad_weight=torch.empty(v, d, dtype=kind, device="cuda"))
        check_backward(dx, dw, x, w, t, lse, rw)


@pytest.mark.parametrize("n", [5, 600])
def test_rows_that_do_not_count(n):
    """Padding, weight 0 and classes past the last: zeros, whatever the rows hold."""
    g = gen(8)
    x, w, t, rw = inputs(g, n, 300, 96, torch.bfloat16, padding=0.0)
    t[0], t[1], t[4] = -1, 300, -5
    rw[2] = 0
    x[0], x[1, 3], x[2] = math.nan, math.inf, -math.inf
    loss, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    with pytest.raises(LoptError):
        L.check_indices()
    assert not bool(loss[[0, 1, 2, 4]].any())
    live = torch.tensor([k not in (0, 1, 2, 4) for k in range(n)], device="cuda")
    check_forward((loss[live], lse[live]), x[live], w, t[live], rw[live])
    for kind in (torch.float32, torch.bfloat16):
        dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw,
                                                 grad_weight=torch.empty(300, 96, dtype=kind, device="cuda"))
        assert not bool(dx[~live].any())
        check_backward(dx[live], dw, x[live], w, t[live], lse[live], rw[live])
    with pytest.raises(LoptError):
        L.check_indices()
    # All of them.
    t[:] = -1
    loss, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw)
    assert not bool(loss.any()) and not bool(dx.any()) and not bool(dw.any())
    L.check_indices()


@pytest.mark.parametrize("d,extra,shift", [(64, 8, 8), (64, 3, 1), (33, 0, 0), (96, 0, 4)])
def test_strides_offsets_and_guards(d, extra, shift):
    g = gen(d)
    n, v, dtype = 70, 333, torch.float16
    x, w, t, rw = inputs(g, n, v, d, dtype)
    px, pw = padded(x, extra, shift, 7.0)[0], padded(w, extra, shift, 7.0)[0]
    (loss, a), (lse, b) = guarded((n,), torch.float32), guarded((n,), torch.float32)
    L.linear_cross_entropy_forward(px, pw, t, row_weight=rw, loss=loss, lse=lse)
    check_forward((loss, lse), x, w, t, rw)
    for kind in (torch.float32, dtype):
        (dx, c), (dw, e) = guarded((n, d), dtype, shift), guarded((v, d), kind, shift)
        L.linear_cross_entropy_backward(px, pw, t, lse, row_weight=rw, grad_x=dx, grad_weight=dw)
        check_backward(dx, dw, x, w, t, lse, rw)
        for whole in (a, b, c, e):
            whole()
    # A gradient that is a block of columns of a wider buffer, more rows than the split form wants.
    x, w, t, rw = inputs(g, 700, v, d, dtype)
    loss, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    wide = torch.full((v, d + 24), 5.0, device="cuda")
    dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, grad_weight=wide[:, 8:8 + d])
    check_backward(dx, dw, x, w, t, lse, rw)
    assert bool((wide[:, :8] == 5).all()) and bool((wide[:, 8 + d:] == 5).all())


def test_one_row_of_x_for_all_and_leading_dimensions():
    g = gen(5)
    x, w, t, rw = inputs(g, 6, 300, 64, torch.bfloat16, padding=0)
    one = x[:1].expand(6, 64)
    check_forward(L.linear_cross_entropy_forward(one, w, t), one, w, t, None)
    loss, lse = L.linear_cross_entropy_forward(x.view(2, 3, 64), w, t.view(2, 3), row_weight=rw.view(2, 3))
    assert loss.shape == lse.shape == (2, 3)
    dx, dw = L.linear_cross_entropy_backward(x.view(2, 3, 64), w, t.view(2, 3), lse, row_weight=rw.view(2, 3))
    assert dx.shape == (2, 3, 64)
    check_backward(dx.view(6, 64), dw, x, w, t, lse.view(6), rw)


@pytest.mark.parametrize("n", [40, 900])
def test_accumulate_parts_and_no_rows(n):
    g = gen(6)
    x, w, t, rw = inputs(g, n, 500, 72, torch.bfloat16)
    _, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw)
    old = normal(g, 500, 72)
    acc = old.clone()
    L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, grad_weight=acc, accumulate=True)
    # With P the tensor cores' sum and H the targets' share, added in one piece per class
    # or a few, acc = (old + P) + H and dw = P + H: each addition is off by half a step
    # of a sum that is at most |old| + |P| + |H|, and |P|, |H| <= the sum of |G| |x| (which
    # P + H may be far below).
    _, _, big = R.ce_backward(x, w, t, lse, rw)
    R.within(acc, old.double() + dw.double(), 8, old.abs().double() + big.abs().t() @ x.double().abs(), "accumulate")
    only = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, need_weight=False)
    assert only[1] is None and float((only[0].double() - dx.double()).abs().max()) <= 2 ** -7 * float(dx.abs().max())
    only = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, need_x=False)
    assert only[0] is None and torch.equal(only[1], dw)
    none, gw = x[:0], torch.ones(500, 72, device="cuda")
    loss, lse = L.linear_cross_entropy_forward(none, w, t[:0])
    assert loss.shape == (0,)
    L.linear_cross_entropy_backward(none, w, t[:0], lse, grad_weight=gw, accumulate=True)
    assert bool((gw == 1).all())
    L.linear_cross_entropy_backward(none, w, t[:0], lse, grad_weight=gw)
    assert not bool(gw.any())


def test_the_same_bits_and_no_leftovers():
    """Two calls give the same bits, also when the workspace held NaN."""
    g = gen(7)
    x, w, t, rw = inputs(g, 700, 3000, 136, torch.float16)
    loss, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    want = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw)
    from learned_optimizer_step_gb300 import train_ops
    for buf, _, _ in train_ops._workspaces.values():
        buf.fill_(255)
    again = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    for buf, _, _ in train_ops._workspaces.values():
        buf.fill_(255)
    assert all(map(torch.equal, want, L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw)))


def test_large_and_small_weights_of_rows():
    """Gradients scale with row_weight, from 1e-30 to 1e30 and below zero."""
    g = gen(9)
    x, w, t, _ = inputs(g, 200, 400, 64, torch.bfloat16)
    _, lse = L.linear_cross_entropy_forward(x, w, t)
    for scale in (1e-30, 1e30, -3.0):
        rw = torch.full((200,), scale, device="cuda")
        dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw)
        rx, rd, _ = R.ce_backward(x, w, t, lse, rw)
        assert float((dw.double() - rd).norm()) <= 2e-5 * float(rd.norm())
        assert float((dx.double() - rx).norm()) <= 2 ** -7 * float(rx.norm())


@pytest.mark.parametrize("dtype", HALF, ids=ids)
def test_targets_that_are_nearly_certain(dtype):
    """Losses from 10 to 1e-10 and what is left of G where they are small, to a relative
    2^-13: a loss is a sum of exponentials of the others' logits, each off by their errors
    (up to 100 half steps and the logits' size, here below 40, times 30 units)."""
    g = gen(12)
    v, d = 300, 64
    w = normal(g, v, d, dtype=dtype, std=0.125)
    t = torch.arange(40, device="cuda")
    x = (normal(g, 40, d, std=0.5) + torch.linspace(0, 30, 40, device="cuda")[:, None] * w[t].float()).to(dtype)
    loss, lse = L.linear_cross_entropy_forward(x, w, t)
    z = x.double() @ w.double().t()
    rest = z.clone()
    rest[torch.arange(40, device="cuda"), t] = -math.inf
    want = torch.nn.functional.softplus(torch.logsumexp(rest, 1) - z[torch.arange(40, device="cuda"), t], threshold=1e9)
    assert float(want.min()) < 1e-5 < 1 < float(want.max())
    assert float(((loss.double() - want) / want).abs().max()) <= 2 ** -13
    exact = torch.logsumexp(z, 1)
    dx, dw = L.linear_cross_entropy_backward(x[:16], w, t[:16], lse[:16])
    _, rd, _ = R.ce_backward(x[:16], w, t[:16], lse[:16], None)
    assert float((dw.double() - rd).norm()) <= 4e-6 * float(rd.norm())
    for k in range(40):          # one token: its own small gradient
        _, dw = L.linear_cross_entropy_backward(x[k:k + 1], w, t[k:k + 1], exact[k:k + 1].float())
        _, rd, _ = R.ce_backward(x[k:k + 1], w, t[k:k + 1], exact[k:k + 1].float(), None)
        assert float((dw.double() - rd).norm()) <= 2 ** -13 * float(rd.norm()), k


def test_infinite_logits():
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(600, 16, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    w[5, 0] = -math.inf           # logit -inf: probability 0
    t = torch.tensor([0, 5, 7, -1], device="cuda")
    loss, lse = L.linear_cross_entropy_forward(x, w, t)
    # The other columns of x are 0, and 0 * 0 = 0: 599 classes at logit 0.
    assert float((lse - math.log(599)).abs().max()) < 1e-5
    assert float(loss[1]) == math.inf and float(loss[3]) == 0 and float(loss[0]) == pytest.approx(math.log(599), rel=1e-6)
    w[6, 0] = math.inf
    loss, lse = L.linear_cross_entropy_forward(x, w, t)
    assert bool(torch.isnan(lse).all() | torch.isinf(lse).all()) and float(loss[3]) == 0


def test_gradients_against_differences():
    """The reference's gradients are the derivative of its losses (float64)."""
    g = torch.Generator()
    g.manual_seed(1)
    x, w = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((5, 7), (11, 7)))
    t, rw = torch.tensor([0, 3, -1, 10, 3]), torch.rand(5, generator=g, dtype=torch.float64)
    _, lse, _ = R.ce_forward(x, w, t, rw)
    dx, dw, _ = R.ce_backward(x, w, t, lse, rw)
    total = lambda a, b: R.ce_forward(a, b, t, rw)[0].sum()   # noqa: E731
    u, v = torch.randn(5, 7, generator=g, dtype=torch.float64), torch.randn(11, 7, generator=g, dtype=torch.float64)
    slope = (total(x + 1e-6 * u, w + 1e-6 * v) - total(x - 1e-6 * u, w - 1e-6 * v)) / 2e-6
    assert abs(float(slope - (dx * u).sum() - (dw * v).sum())) < 1e-7


def test_refusals():
    g = gen(1)
    x, w, t, rw = inputs(g, 6, 50, 32, torch.bfloat16)
    _, lse = L.linear_cross_entropy_forward(x, w, t)
    F, B = L.linear_cross_entropy_forward, L.linear_cross_entropy_backward
    gw = torch.zeros(50, 32, device="cuda")
    for call, error in ((lambda: F(x.float(), w.float(), t), TypeError), (lambda: F(x, w.half(), t), TypeError),
                        (lambda: F(x, w[:, :16], t), ValueError), (lambda: F(x, w.t(), t), ValueError),
                        (lambda: F(x, w, t[:3]), ValueError), (lambda: F(x, w, t.float()), TypeError),
                        (lambda: F(x, w, t, row_weight=rw.half()), TypeError), (lambda: F(x.cpu(), w, t), TypeError),
                        (lambda: F(x, w, t, loss=lse, lse=lse), LoptError),
                        (lambda: B(x, w, t, lse[:2]), ValueError), (lambda: B(x, w, t, None), TypeError),
                        (lambda: B(x, w, t, lse, grad_x=x), LoptError),
                        (lambda: B(x, w, t, lse, grad_weight=w), LoptError),
                        (lambda: B(x, w, t, lse, grad_weight=gw.half()), TypeError),
                        (lambda: B(x, w, t, lse, accumulate=True), ValueError),
                        (lambda: B(x, w, t, lse, grad_weight=gw.bfloat16(), accumulate=True), TypeError),
                        (lambda: B(x, w, t, lse, grad_weight=gw[:10]), ValueError),
                        (lambda: F(x.clone().requires_grad_(), w, t), RuntimeError)):
        with pytest.raises(error):
            call()
