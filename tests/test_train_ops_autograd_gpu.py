"""The training operators beside autograd on the GPU: what it would have to
record is refused, and what they write counts as changed."""

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import distill_inputs, gen, norm_inputs, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def calls():
    """Per operator: the call, its tensors that may require a gradient, those that it writes."""
    g = gen(1)
    x, w, b = norm_inputs(g, 6, 64, torch.float32, torch.float32)
    r, dy, table = normal(g, 6, 64), normal(g, 6, 64), normal(g, 20, 64)
    index = torch.randint(0, 20, (6,), generator=g, device="cuda")
    z, t, i = distill_inputs(g, 6, 64, 4, torch.float32, torch.float32, torch.int64)
    rw = torch.ones(6, device="cuda")
    e = lambda *shape: torch.zeros(*shape, device="cuda")   # noqa: E731
    o, m, v = [e(6, 64) for _ in range(4)], e(6), e(6) + 1
    gw, gb, gt, loss = e(64), e(64), e(20, 64), e(6)
    return [
        (lambda: L.embedding_forward(table, index, out=o[0]), [table], [o[0]]),
        (lambda: L.embedding_backward(dy, index, 20, out=gt), [dy], [gt]),
        (lambda: L.layernorm_forward(x, w, b, residual=r, out=o[1], summed=o[2], mean=m, rstd=v), [x, w, b, r],
         [o[1], o[2], m, v]),
        (lambda: L.layernorm_backward(dy, x, m, v, w, grad_residual=r, grad_x=o[3], grad_weight=gw, grad_bias=gb),
         [dy, x, w, r], [o[3], gw, gb]),
        (lambda: L.distill_forward(z, t, i, row_weight=rw, loss=loss), [z, t, rw], [loss]),
        (lambda: L.distill_forward_backward(z, t, i, row_weight=rw, loss=loss, grad=z), [z, t, rw], [loss, z]),
    ]


@pytest.mark.parametrize("k", range(6))
def test_tensors_that_require_a_gradient_are_refused(k):
    call, inputs, _ = calls()[k]
    call()
    for t in inputs:
        t.requires_grad_()
        with pytest.raises(RuntimeError, match="not recorded by autograd"):
            call()
        with torch.no_grad():
            call()
        t.requires_grad_(False)


@pytest.mark.parametrize("k", range(6))
def test_written_tensors_count_as_changed(k):
    call, inputs, written = calls()[k]
    before = [t._version for t in written]
    read = [(t, t._version) for t in inputs if all(t is not o for o in written)]
    call()
    assert all(t._version > v for t, v in zip(written, before))
    assert all(t._version == v for t, v in read)


def test_autograd_notices_an_overwritten_tensor():
    p = torch.ones(6, 64, device="cuda", requires_grad=True)
    y = p.exp()                                   # saves y
    w = torch.ones(64, device="cuda")
    L.layernorm_forward(torch.ones(6, 64, device="cuda"), w, out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_from_an_autograd_function():
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            y, mean, rstd = L.layernorm_forward(x, w, b)
            ctx.save_for_backward(x, w, mean, rstd)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, w, mean, rstd = ctx.saved_tensors
            return L.layernorm_backward(dy, x, mean, rstd, w)
    g = gen(2)
    x, w, b = norm_inputs(g, 6, 64, torch.float32, torch.float32)
    dy = normal(g, 6, 64)
    _, mean, rstd = L.layernorm_forward(x, w, b)
    want = L.layernorm_backward(dy, x, mean, rstd, w)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    Norm.apply(*leaves).backward(dy)
    assert all(torch.equal(t.grad, v) for t, v in zip(leaves, want))
