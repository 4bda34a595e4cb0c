"""The training operators' kernels on the GPU, against plain float64 forms
(tests/train_reference.py) with bounds derived from the roundings, at the
sizes, strides and masks where they can go wrong."""

import math

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from learned_optimizer_step_gb300 import LoptError
from learned_optimizer_step_gb300 import train_ops as ops
from tests import train_reference as R
from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
ids = lambda v: str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None   # noqa: E731


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def padded(t, extra, shift=0, fill=math.nan):
    """The same matrix with `extra` more elements between rows, `shift`
    elements into its buffer; the rest holds `fill`."""
    rows, cols = t.shape
    buf = torch.full((shift + rows * (cols + extra) + 64,), fill, dtype=t.dtype, device="cuda")
    v = buf[shift:shift + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
    v.copy_(t)
    return v, buf


def guarded(shape, dtype, shift=0):
    """An output tensor between guard zones, and a check that they are whole."""
    n = math.prod(shape)
    buf = torch.full((shift + n + 256,), -77.0, dtype=dtype, device="cuda")
    t = buf[128 + shift:128 + shift + n].view(shape)

    def whole():
        assert bool((buf[:128 + shift] == -77.0).all()) and bool((buf[128 + shift + n:] == -77.0).all()), "guard zone"
    return t, whole


# ---- embedding ------------------------------------------------------------------


@pytest.mark.parametrize("table_dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("out_dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (5, 7, 8), (33, 100, 768), (257, 1000, 435), (64, 300, 2048),
                                         (3, 50, 4104)])
def test_embedding_forward(table_dtype, out_dtype, n, rows, cols):
    g = gen(n + cols)
    table = normal(g, rows, cols, dtype=table_dtype)
    for it in (torch.int32, torch.int64):
        index = torch.randint(-1, rows, (n,), generator=g, device="cuda").to(it)
        out, whole = guarded((n, cols), out_dtype)
        assert L.embedding_forward(table, index, 1.5, out=out) is out
        want = torch.where((index >= 0)[:, None], table[index.long().clamp(min=0)].float() * 1.5, 0.0).to(out_dtype)
        assert torch.equal(out, want)   # one product, one rounding
        whole()


def test_embedding_forward_strides_shapes_and_new_output():
    g = gen(1)
    table = normal(g, 40, 96)
    wide, _ = padded(table, 7, 3)
    index = torch.randint(0, 40, (3, 5), generator=g, device="cuda")
    out = L.embedding_forward(wide, index, out_dtype=torch.bfloat16)
    assert out.shape == (3, 5, 96) and out.dtype == torch.bfloat16
    assert torch.equal(out, table[index].bfloat16())
    buf = torch.full((15, 200), 9.0, device="cuda")
    L.embedding_forward(table, index.view(-1), out=buf[:, 10:106])
    assert torch.equal(buf[:, 10:106], table[index.view(-1)])
    assert bool((buf[:, :10] == 9).all()) and bool((buf[:, 106:] == 9).all())
    empty = L.embedding_forward(table, index.view(-1)[:0])
    assert empty.shape == (0, 96)


@pytest.mark.parametrize("index_dtype", [torch.int32, torch.int64], ids=ids)
def test_bad_indices_are_reported(index_dtype):
    ops.check_indices()
    table = torch.ones(10, 16, device="cuda")
    index = torch.tensor([3, 10, -1, 9], device="cuda", dtype=index_dtype)
    out = L.embedding_forward(table, index)
    assert out[:, 0].tolist() == [1, 0, 0, 1]
    with pytest.raises(LoptError) as e:
        L.check_indices()
    assert e.value.code == ops.E_INDEX
    L.check_indices()                                # reported once
    grad = L.embedding_backward(torch.ones(4, 16, device="cuda"), index, 10)
    assert grad.sum(1).tolist() == [0, 0, 0, 16, 0, 0, 0, 0, 0, 16]
    with pytest.raises(LoptError):
        L.check_indices()
    if index_dtype is torch.int64:                   # beyond 32 bits
        L.embedding_forward(table, torch.tensor([1 << 40, (1 << 32) + 3], device="cuda"))
        with pytest.raises(LoptError):
            L.check_indices()
        lost = L.embedding_backward(torch.ones(2, 16, device="cuda"), torch.tensor([(1 << 32) + 3, -(1 << 40)], device="cuda"), 10)
        assert not lost.any()
        with pytest.raises(LoptError):
            L.check_indices()


def token_lists(g, n, rows):
    """Index lists that stress the sort and the runs: text-like, all equal,
    all different, all padding, one hot token among rare ones."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    yield "text", (torch.exp(u * math.log(rows + 1.0)) - 1).long().clamp(0, rows - 1)
    yield "equal", torch.full((n,), rows - 1, device="cuda")
    yield "different", torch.randperm(max(n, rows), generator=g, device="cuda")[:n] % rows
    yield "padding", torch.full((n,), -1, device="cuda")
    hot = torch.randint(-1, rows, (n,), generator=g, device="cuda")
    hot[torch.rand(n, generator=g, device="cuda") < 0.6] = rows // 2
    yield "hot", hot


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (1, 5, 8), (7, 3, 24), (8, 9, 16), (31, 64, 100), (300, 50, 435),
                                         (1025, 1500, 72), (4099, 257, 768), (20000, 3001, 40), (70, 40, 4104)])
def test_embedding_backward(dtype, n, rows, cols):
    g = gen(n * 31 + cols)
    for k, (kind, index) in enumerate(token_lists(g, n, rows)):
        dy = normal(g, n, cols, dtype=dtype)
        index = index.to(torch.int32 if k % 2 else torch.int64)
        want, bound = R.embed_backward(dy, index, rows, 0.75)
        out, whole = guarded((rows, cols), torch.float32)
        L.embedding_backward(dy, index, rows, 0.75, out=out)
        R.check(out, want, bound, kind)
        whole()
        again = L.embedding_backward(dy, index, rows, 0.75)
        assert torch.equal(out, again), kind           # the same bits
        base = normal(g, rows, cols)
        acc = base.clone()
        L.embedding_backward(dy, index, rows, 0.75, out=acc, accumulate=True)
        R.check(acc, base.double() + want, bound + R.u * (base.double().abs() + want.abs()) * 1.01, kind + " accumulated")


def test_embedding_backward_ignores_masked_rows_and_takes_strides():
    g = gen(5)
    dy = normal(g, 50, 64, dtype=torch.bfloat16)
    index = torch.randint(0, 20, (50,), generator=g, device="cuda")
    want, bound = R.embed_backward(dy, index, 20, 1.0)
    for extra, shift in ((8, 0), (3, 1), (0, 1)):
        v, _ = padded(dy, extra, shift)
        R.check(L.embedding_backward(v, index, 20), want, bound, "stride")
    one = dy[:1].expand(50, 64)                        # the gradient of a broadcast sum
    want1, bound1 = R.embed_backward(one, index, 20, 1.0)
    R.check(L.embedding_backward(one, index, 20), want1, bound1, "broadcast")
    masked = dy.clone()
    masked[::3] = math.nan
    skipped = index.clone()
    skipped[::3] = -1
    want, bound = R.embed_backward(dy, skipped, 20, 1.0)
    R.check(L.embedding_backward(masked, skipped, 20), want, bound, "NaN under the mask")
    buf = torch.full((23,), 5.0, device="cuda")
    odd = buf[1:21].view(20, 1)                        # a gradient buffer off the 16-byte boundary
    L.embedding_backward(dy[:, :1], index, 20, out=odd)
    want, bound = R.embed_backward(dy[:, :1], index, 20, 1.0)
    R.check(odd, want, bound, "misaligned")
    assert buf[0] == 5 and bool((buf[21:] == 5).all())


def test_embedding_backward_without_tokens():
    dy, index = torch.ones(0, 8, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    out = torch.full((4, 8), 3.0, device="cuda")
    L.embedding_backward(dy, index, 4, out=out, accumulate=True)
    assert bool((out == 3).all())
    L.embedding_backward(dy, index, 4, out=out)
    assert not out.any()


def test_embedding_pair_is_a_gradient():
    """<dW, V> equals the change of <out, dy> along V: the lookup is linear,
    so a difference of any step gives it up to rounding."""
    g = gen(9)
    W, V = normal(g, 60, 48), normal(g, 60, 48)
    index = torch.randint(-1, 60, (500,), generator=g, device="cuda")
    dy = normal(g, 500, 48)
    dW = L.embedding_backward(dy, index, 60, 2.0)
    f = lambda t: (L.embedding_forward(t, index, 2.0).double() * dy.double()).sum()   # noqa: E731
    diff = f(W + V) - f(W - V)
    slope = 2 * (dW.double() * V.double()).sum()
    mag = (L.embedding_forward(W.abs() + V.abs(), index, 2.0).double() * dy.double().abs()).sum()
    assert abs(float(diff - slope)) <= 600 * R.u * float(mag)


# ---- layer norm --------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (3, 2), (5, 8), (9, 100), (17, 256), (4, 435), (33, 768), (2, 1000), (7, 1024), (6, 2048),
               (3, 4104), (5, 5001), (2, 8192), (3, 16384), (2, 16392), (1, 20001)]


def norm_inputs(g, rows, cols, dtype, wt):
    x = (torch.randn(rows, cols, generator=g, device="cuda")
         * torch.exp(torch.randn(cols, generator=g, device="cuda") * 0.5) + 0.3).to(dtype)
    return x, normal(g, cols, dtype=wt, std=0.2, mean=1.0), normal(g, cols, dtype=wt, std=0.2)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_layernorm_forward(dtype, rows, cols):
    g = gen(rows + cols)
    for wt in {torch.float32, dtype}:
        x, w, b = norm_inputs(g, rows, cols, dtype, wt)
        for residual in (None, normal(g, rows, cols, dtype=dtype)):
            for bias in (b, None):
                y, sm, mean, rstd = R.norm_forward(x, w, bias, 1e-5, residual)
                by, bs, bm, br = R.norm_forward_bounds(sm, mean, rstd, y, w, bias, dtype)
                out, whole = guarded((rows, cols), dtype)
                got = L.layernorm_forward(x, w, bias, 1e-5, residual=residual, out=out)
                assert got[0] is out and len(got) == (3 if residual is None else 4)
                R.check(got[0], y, by, "y")
                R.check(got[-2], mean, bm, "mean")
                R.check(got[-1], rstd, br, "rstd")
                if residual is not None:
                    assert torch.equal(got[1], (x.float() + residual.float()).to(dtype))
                whole()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(2047, 96), (4000, 33), (700, 768)])
def test_layernorm_backward(dtype, rows, cols):
    g = gen(3 * rows + cols)
    for wt in {torch.float32, dtype}:
        x, w, _ = norm_inputs(g, rows, cols, dtype, wt)
        dy = normal(g, rows, cols, dtype=dtype)
        _, _, mean, rstd = R.norm_forward(x, w, None, 1e-5)
        mean, rstd = mean.float(), rstd.float()
        for dres in (None, normal(g, rows, cols, dtype=dtype)):
            dx, dw, db = R.norm_backward(dy, x, mean, rstd, w, dres)
            bx, bw, bb = R.norm_backward_bounds(dy, x, mean, rstd, w, dx, dtype, dres)
            out, whole = guarded((rows, cols), dtype)
            gw, whole_w = guarded((cols,), torch.float32, 1)
            gb, whole_b = guarded((cols,), torch.float32, 1)
            got = L.layernorm_backward(dy, x, mean, rstd, w, grad_residual=dres, grad_x=out, grad_weight=gw,
                                       grad_bias=gb)
            R.check(got[0], dx, bx, "dx")
            R.check(got[1], dw, bw, "dweight")
            R.check(got[2], db, bb, "dbias")
            whole(), whole_w(), whole_b()
            again = L.layernorm_backward(dy, x, mean, rstd, w, grad_residual=dres, need_bias=False)
            assert again[2] is None and torch.equal(again[0], out) and torch.equal(again[1], gw)
        base = normal(g, cols)
        aw, ab = base.clone(), base.clone()
        L.layernorm_backward(dy, x, mean, rstd, w, grad_weight=aw, grad_bias=ab, accumulate=True)
        assert torch.equal(aw, base + gw) and torch.equal(ab, base + gb)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("cols", [768, 435, 2048, 20001])
def test_layernorm_strides_and_in_place(dtype, cols):
    g = gen(cols)
    rows = 11
    x, w, b = norm_inputs(g, rows, cols, dtype, torch.float32)
    r, dy, dr = (normal(g, rows, cols, dtype=dtype) for _ in range(3))
    base = L.layernorm_forward(x, w, b, residual=r)
    back = L.layernorm_backward(dy, base[1], base[2], base[3], w, grad_residual=dr)
    for extra, shift in ((8, 0), (3, 1), (0, 1)):
        xs, rs, dys, drs = (padded(t, extra, shift)[0] for t in (x, r, dy, dr))
        ys, ybuf = padded(torch.zeros_like(x), extra, shift, 7.0)
        got = L.layernorm_forward(xs, w, b, residual=rs, out=ys)
        by = R.norm_forward_bounds(*_spread(R.norm_forward(x, w, b, 1e-5, r)), w, b, dtype)
        for a, c, bound in zip(got, R.norm_forward(x, w, b, 1e-5, r), by):
            R.check(a, c, bound, "strided")
        assert int((ybuf == 7.0).sum()) >= ybuf.numel() - x.numel()   # nothing between the rows is written
        gb = L.layernorm_backward(dys, padded(base[1], extra, shift)[0], base[2], base[3], w, grad_residual=drs)
        dx, dw, db = R.norm_backward(dy, base[1], base[2], base[3], w, dr)
        bounds = R.norm_backward_bounds(dy, base[1], base[2], base[3], w, dx, dtype, dr)
        for a, c, bound in zip(gb, (dx, dw, db), bounds):
            R.check(a, c, bound, "strided backward")
    xi, ri = x.clone(), r.clone()
    L.layernorm_forward(xi, w, b, residual=ri, out=xi, summed=ri)
    assert torch.equal(xi, base[0]) and torch.equal(ri, base[1])
    for which in range(3):
        t = [dy.clone(), base[1].clone(), dr.clone()]
        got = L.layernorm_backward(t[0], t[1], base[2], base[3], w, grad_residual=t[2], grad_x=t[which])
        assert torch.equal(got[0], back[0]) and torch.equal(got[1], back[1]) and torch.equal(got[2], back[2])


def _spread(fwd):
    y, s, mean, rstd = fwd
    return s, mean, rstd, y


def test_layernorm_rows_of_one_value_far_means_and_nan():
    w, b = torch.ones(256, device="cuda"), torch.zeros(256, device="cuda")
    x = torch.full((4, 256), 3.0, device="cuda")
    x[1] = 1e4 + torch.arange(256, device="cuda") * 0.01     # spread far below the mean
    x[2, 7] = math.nan
    x[3, 9] = math.inf
    y, mean, rstd = L.layernorm_forward(x, w, b, 1e-5)
    assert not y[0].any() and abs(float(rstd[0]) - 1e5 ** 0.5) < 1e-3 * 1e5 ** 0.5
    want = R.norm_forward(x[1:2], w, b, 1e-5)
    bounds = R.norm_forward_bounds(want[1], want[2], want[3], want[0], w, b, torch.float32)
    R.check(y[1:2], want[0], bounds[0], "far mean")
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()


def test_layernorm_shapes_rows_zero_and_broadcast_gradient():
    g = gen(2)
    x, w, b = norm_inputs(g, 30, 64, torch.bfloat16, torch.float32)
    y, mean, rstd = L.layernorm_forward(x.view(2, 3, 5, 64), w, b)
    assert y.shape == (2, 3, 5, 64) and mean.shape == (2, 3, 5)
    flat = L.layernorm_forward(x, w, b)
    assert torch.equal(y.view(30, 64), flat[0])
    dy = normal(g, 1, 64, dtype=torch.bfloat16).expand(30, 64)
    got = L.layernorm_backward(dy, x, flat[1], flat[2], w)
    again = L.layernorm_backward(dy.contiguous(), x, flat[1], flat[2], w)
    assert all(torch.equal(a, c) for a, c in zip(got, again))
    e = x[:0]
    y, mean, rstd = L.layernorm_forward(e, w, b)
    assert y.shape == (0, 64) and mean.shape == (0,)
    gw, gb = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    L.layernorm_backward(e, e, mean, rstd, w, grad_weight=gw, grad_bias=gb, accumulate=True)
    assert bool((gw == 1).all())
    L.layernorm_backward(e, e, mean, rstd, w, grad_weight=gw, grad_bias=gb)
    assert not gw.any() and not gb.any()


def test_layernorm_backward_is_the_gradient_by_differences():
    g = gen(4)
    rows, cols = 6, 200
    x, w, b = norm_inputs(g, rows, cols, torch.float32, torch.float32)
    dy = normal(g, rows, cols)
    _, mean, rstd = L.layernorm_forward(x, w, b)
    grads = L.layernorm_backward(dy, x, mean, rstd, w)

    def f(x, w, b):
        return float((L.layernorm_forward(x, w, b)[0].double() * dy.double()).sum())
    h = 2.0 ** -6
    mag = float((L.layernorm_forward(x, w, b)[0].double().abs() * dy.double().abs()).sum())
    for k, t in enumerate((x, w, b)):
        v = normal(g, *t.shape)
        plus, minus = [x, w, b], [x, w, b]
        plus[k], minus[k] = t + h * v, t - h * v
        diff = (f(*plus) - f(*minus)) / (2 * h)
        slope = float((grads[k].double() * v.double()).sum())
        exact = [R.norm_forward(p[0], p[1], p[2], 1e-5)[0] for p in (plus, minus)]
        true = float(((exact[0] - exact[1]) * dy.double()).sum()) / (2 * h)
        step = abs(true - float((R_grads(dy, x, w)[k] * v.double()).sum()))     # the difference's own error
        noise = 16 * R.u * mag / h + 200 * R.u * float((grads[k].double().abs() * v.double().abs()).sum())
        assert abs(diff - slope) <= step + noise, k


def R_grads(dy, x, w):
    _, _, mean, rstd = R.norm_forward(x, w, None, 1e-5)
    return R.norm_backward(dy, x, mean, rstd, w)


# ---- distillation --------------------------------------------------------------------


def distill_inputs(g, rows, cols, top, dtype, tt, it):
    z = normal(g, rows, cols, dtype=dtype, std=3.0)
    teacher = z.float() * 0.7 + normal(g, rows, cols, std=1.5)
    t, i = torch.topk(teacher, min(top, cols), 1)
    if top > cols:                                       # more slots than classes: repeats
        more = torch.randint(0, cols, (rows, top - cols), generator=g, device="cuda")
        t, i = torch.cat([t, teacher.gather(1, more)], 1), torch.cat([i, more], 1)
    i = torch.where(torch.rand(rows, top, generator=g, device="cuda") < 0.2, -1, i)
    return z, t.to(tt), i.to(it)


def check_distill(z, t, i, T, w, got_loss, got_grad, what):
    loss, grad = R.distill(z, t, i, T, w)
    b_loss, b_grad = R.distill_bounds(z, t, i, T, grad, w)
    R.check(got_loss, loss, b_loss, what + " loss")
    if got_grad is not None:
        R.check(got_grad, grad, b_grad + R.rounded(grad, z.dtype) * 1.01, what + " grad")


DISTILL_SHAPES = [(1, 1, 1), (3, 2, 1), (5, 7, 9), (4, 100, 16), (9, 257, 20), (33, 1000, 20), (2, 4096, 64),
                  (3, 5003, 33), (2, 16001, 128), (3, 50257, 64), (2, 50304, 1024), (2, 131072, 17), (1, 262147, 3)]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("rows,cols,top", DISTILL_SHAPES)
def test_distill(dtype, rows, cols, top):
    g = gen(rows + cols + top)
    for tt, it, T in ((torch.float32, torch.int64, 1.0), (dtype, torch.int32, 2.5)):
        z, t, i = distill_inputs(g, rows, cols, top, dtype, tt, it)
        w = torch.rand(rows, generator=g, device="cuda") + 0.5
        if rows > 2:
            w[1] = 0.0
        grad, whole = guarded((rows, cols), dtype)
        loss, whole_l = guarded((rows,), torch.float32, 1)
        got = L.distill_forward_backward(z, t, i, T, row_weight=w, loss=loss, grad=grad)
        assert got[0] is loss and got[1] is grad
        check_distill(z, t, i, T, w, loss, grad, "T=%g" % T)
        whole(), whole_l()
        assert torch.equal(L.distill_forward(z, t, i, T, row_weight=w), loss)
        zi = z.clone()
        again = L.distill_forward_backward(zi, t, i, T, row_weight=w, grad=zi)   # in place
        assert torch.equal(zi, grad) and torch.equal(again[0], loss)
        check_distill(z, t, i, T, None, *L.distill_forward_backward(z, t, i, T), "no weights")


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("cols", [64, 333, 9001])
def test_distill_strides(dtype, cols):
    g = gen(cols)
    z, t, i = distill_inputs(g, 7, cols, 12, dtype, torch.float32, torch.int64)
    for extra, shift in ((8, 0), (3, 1), (0, 1), (1, 0)):
        for g_extra in (0, extra):
            zs, ts = padded(z, extra, shift)[0], padded(t, 5, 1)[0]
            i_s = padded(i, 3, 0, 99)[0]
            gs, buf = padded(torch.zeros_like(z), g_extra, shift, 7.0)
            loss, grad = L.distill_forward_backward(zs, ts, i_s, 1.5, grad=gs)
            check_distill(z, t, i, 1.5, None, loss, grad, "strided")
            assert int((buf == 7.0).sum()) >= buf.numel() - z.numel()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("cols", [40, 5003, 50257])
def test_distill_masks(dtype, cols):
    """Masked classes (-inf and the type's lowest value), empty rows, teacher
    slots of -inf, repeated classes, weights of zero over NaN logits."""
    g = gen(cols + 1)
    rows, top = 10, 6
    z, t, i = distill_inputs(g, rows, cols, top, dtype, torch.float32, torch.int64)
    i = i.abs()
    low = torch.finfo(dtype).min
    z[0, cols // 2:] = -math.inf
    i[0] = i[0] % (cols // 2)
    z[1, cols // 2:] = low
    i[1] = i[1] % (cols // 2)
    z[2] = low                                   # nothing but masked: all classes alike
    i[3] = -1                                    # no slot
    t[4] = -math.inf                             # slots without probability
    t[5, 1:] = -math.inf                         # one slot: cross entropy
    i[6] = i[6, 0]                               # one class six times
    z[7] = math.nan                              # not counted: not read
    t[8] = torch.finfo(torch.float32).min        # all slots at the lowest value: equal
    z[9, 3] = -math.inf                          # the teacher wants a masked class
    i[9, 0] = 3
    w = torch.ones(rows, device="cuda")
    w[7] = 0.0
    loss, grad = L.distill_forward_backward(z, t, i, 2.0, row_weight=w)
    want_l, want_g = R.distill(torch.nan_to_num(z, nan=0.0, posinf=math.inf, neginf=-math.inf), t, i, 2.0, w)
    b_l, b_g = R.distill_bounds(torch.nan_to_num(z, nan=0.0, posinf=math.inf, neginf=-math.inf), t, i, 2.0, want_g, w)
    R.check(loss, want_l, torch.nan_to_num(b_l, nan=0.0, posinf=0.0), "loss")
    R.check(grad, want_g, b_g + R.rounded(want_g, dtype) * 1.01, "grad")
    assert loss[9] == math.inf and not loss[[3, 4, 7]].any() and not grad[[3, 4, 7]].any()
    nan = z.clone()
    nan[0, 1] = math.nan
    loss, grad = L.distill_forward_backward(nan, t, i, 2.0, row_weight=w)
    assert math.isnan(loss[0]) and torch.isnan(grad[0]).all() and torch.isfinite(grad[1]).all()


def test_distill_one_slot_is_cross_entropy():
    g = gen(12)
    z = normal(g, 50, 777, dtype=torch.float32, std=2.0)
    y = torch.randint(0, 777, (50, 1), generator=g, device="cuda")
    loss, grad = L.distill_forward_backward(z, torch.zeros(50, 1, device="cuda"), y)
    logq = torch.log_softmax(z.double(), 1)
    R.check(loss, -logq.gather(1, y)[:, 0], torch.full_like(loss, 400 * R.u, dtype=R.F64), "cross entropy")
    want = logq.exp().scatter_add(1, y, torch.full((50, 1), -1.0, dtype=R.F64, device="cuda"))
    R.check(grad, want, torch.full_like(want, 100 * R.u), "its gradient")


def test_distill_bad_indices_and_empty_batch():
    ops.check_indices()
    z = torch.zeros(2, 10, device="cuda")
    t = torch.zeros(2, 3, device="cuda")
    i = torch.tensor([[1, 10, -5], [1 << 40, 10, 11]], device="cuda")
    loss, grad = L.distill_forward_backward(z, t, i)
    assert abs(float(loss[0]) - math.log(10)) < 1e-5 and loss[1] == 0 and not grad[1].any()
    with pytest.raises(LoptError):
        L.check_indices()
    loss, grad = L.distill_forward_backward(z[:0], t[:0], i[:0])
    assert loss.shape == (0,) and grad.shape == (0, 10)


def test_distill_gradient_by_differences():
    g = gen(21)
    z, t, i = distill_inputs(g, 4, 300, 10, torch.float32, torch.float32, torch.int64)
    v = normal(g, 4, 300)
    h = 2.0 ** -6
    _, grad = L.distill_forward_backward(z, t, i, 2.0)
    f = lambda a: L.distill_forward(a, t, i, 2.0).double()      # noqa: E731
    diff = (f(z + h * v) - f(z - h * v)) / (2 * h)
    slope = (grad.double() * v.double()).sum(1)
    true = (R.distill(z + h * v, t, i, 2.0)[0] - R.distill(z - h * v, t, i, 2.0)[0]) / (2 * h)
    step = (true - (R.distill(z, t, i, 2.0)[1] * v.double()).sum(1)).abs()
    b_loss, b_grad = R.distill_bounds(z, t, i, 2.0, grad)
    noise = 2 * b_loss / h + ((b_grad + 2 * R.u * grad.double().abs()) * v.double().abs()).sum(1)
    assert bool(((diff - slope).abs() <= step + noise).all())


# ---- calls ---------------------------------------------------------------------------


def test_other_stream_and_graph():
    """A call on another stream than the current one, and a captured one."""
    g = gen(33)
    z, t, i = distill_inputs(g, 64, 5003, 8, torch.bfloat16, torch.float32, torch.int64)
    x, w, b = norm_inputs(g, 64, 768, torch.bfloat16, torch.float32)
    table, index = normal(g, 500, 768), torch.randint(0, 500, (64,), generator=g, device="cuda")

    def everything(stream=None):
        e = L.embedding_forward(table, index, out_dtype=torch.bfloat16, stream=stream)
        y, mean, rstd = L.layernorm_forward(e, w, b, stream=stream)
        loss, grad = L.distill_forward_backward(z, t, i, stream=stream)
        dx, dw, db = L.layernorm_backward(x, e, mean, rstd, w, stream=stream)
        dt = L.embedding_backward(dx, index, 500, stream=stream)
        return [e, y, mean, rstd, loss, grad, dx, dw, db, dt]
    want = everything()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = everything(stream)
        s.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything()
    for a in got:
        a.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_refusals_of_the_binding():
    f = torch.zeros(4, 8, device="cuda")
    i = torch.zeros(4, dtype=torch.int64, device="cuda")
    w = torch.ones(8, device="cuda")
    m = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        L.embedding_forward(f.cpu(), i)
    with pytest.raises(TypeError):
        L.embedding_forward(f, i.cpu())
    with pytest.raises(TypeError):
        L.embedding_forward(f, i.float())
    with pytest.raises(TypeError):
        L.embedding_forward(f.double(), i)
    with pytest.raises(ValueError):
        L.embedding_forward(f, i, out=torch.zeros(4, 9, device="cuda"))
    with pytest.raises(ValueError):
        L.embedding_forward(f.t(), i)
    with pytest.raises(ValueError):
        L.embedding_backward(f, i[:3], 5)
    with pytest.raises(ValueError):
        L.embedding_backward(f, i, 5, accumulate=True)
    with pytest.raises(TypeError):
        L.embedding_backward(f, i, 5, out=torch.zeros(5, 8, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(LoptError):
        L.embedding_backward(f, i, 4, out=f)                    # overlaps
    with pytest.raises(LoptError):
        L.embedding_forward(f, i, out=f)
    with pytest.raises(ValueError):
        L.layernorm_forward(f, w[:7])
    with pytest.raises(TypeError):
        L.layernorm_forward(f, w.half())
    with pytest.raises(ValueError):
        L.layernorm_forward(f, w, summed=f.clone())
    with pytest.raises(LoptError):
        L.layernorm_forward(f, w, eps=-1.0)
    with pytest.raises(LoptError):
        L.layernorm_forward(f, w, mean=m, rstd=m)
    with pytest.raises(LoptError):
        L.layernorm_forward(f[:3], w, out=f[1:])                # overlaps by two rows
    with pytest.raises(LoptError):
        L.layernorm_forward(f, w, out=torch.zeros(8, device="cuda").expand(4, 8))
    with pytest.raises(ValueError):
        L.layernorm_backward(f, f[:3], m, m, w)
    with pytest.raises(ValueError):
        L.layernorm_backward(f, f, m, m, w, accumulate=True)
    with pytest.raises(LoptError):
        L.layernorm_backward(f, f, m, m, w, grad_weight=w)
    i2 = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    t2 = torch.zeros(4, 2, device="cuda")
    with pytest.raises(ValueError):
        L.distill_forward(f, t2, i2[:3])
    with pytest.raises(LoptError):
        L.distill_forward(f, t2, i2, 0.0)
    with pytest.raises(LoptError):
        L.distill_forward(f, t2, i2, math.nan)
    with pytest.raises(LoptError):
        L.distill_forward(f, torch.zeros(4, 1025, device="cuda"), torch.zeros(4, 1025, dtype=torch.int32, device="cuda"))
    with pytest.raises(LoptError):
        L.distill_forward(f, t2[:, :0], i2[:, :0])
    with pytest.raises(TypeError):
        L.distill_forward(f, t2.half(), i2)
    with pytest.raises(LoptError):
        L.distill_forward_backward(f[:3], t2[:3], i2[:3], grad=f[1:])
    # column blocks of one buffer do not overlap
    buf = torch.randn(4, 16, device="cuda")
    x = buf[:, :8].clone()
    L.layernorm_forward(buf[:, :8], w, out=buf[:, 8:])
    assert torch.equal(buf[:, :8], x) and torch.equal(buf[:, 8:], L.layernorm_forward(x, w)[0])
