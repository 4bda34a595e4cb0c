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


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("n,v,d", [(5, 5003, 256), (17, 5003, 256), (64, 5003, 256), (203, 5003, 256), (700, 5003, 256),
                                   (2100, 5003, 101), (700, 20000, 640)])
def test_16_bit_gradients_are_as_exact_as_their_type(n, v, d, dtype):
    """What rounding the exact gradients would leave, 5 % for its being other elements that
    are rounded, 2^-16 for the logits' errors and the second part of G, and, where G has one
    part, half a step of each of its entries but the targets', which are independent: the
    root of the sum of their squares."""
    x, w, t, rw = inputs(gen(n), n, v, d, dtype, padding=0.1)
    _, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    want_x, want_w, g = R.ce_backward(x, w, t, lse, rw)
    others = g.clone()
    others[torch.arange(n, device="cuda"), t.clamp(min=0)] = 0
    half = R.half_step(dtype)
    one_x = half * float(((others ** 2) @ (w.double() ** 2)).sum().sqrt() / want_x.norm()) if n > 16 else 0.0
    one_w = half * float(((others ** 2).t() @ (x.double() ** 2)).sum().sqrt() / want_w.norm()) if n > 512 else 0.0
    assert one_x < 0.1 * half and one_w < 0.1 * half       # else the bound would say nothing
    for kind in (dtype, torch.float32, None):
        gw = None if kind is None else torch.empty(v, d, dtype=kind, device="cuda")
        dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, grad_weight=gw, need_weight=gw is not None)
        assert off(dx, want_x) <= 1.05 * off(want_x.to(dtype), want_x) + 2.0 ** -16 + one_x
        if kind is dtype:
            assert off(dw, want_w) <= 1.05 * off(want_w.to(dtype), want_w) + 2.0 ** -16 + one_w


@pytest.mark.parametrize("dtype", HALF, ids=ids)
def test_long_sums_of_one_sign(dtype):
    """1,048,576 tokens whose terms of grad_weight all have one sign: what the tensor cores
    cut from a sum adds up.  The mean error of the gradients of 63 classes: a sum of 128
    steps of 64 tokens, four products of 16 each, which cut four half steps of float32 at
    most; the sums' own additions, a half step each; and what rounding a class's entries of
    G and its gradients leaves, each up to half a step of the type and evenly spread from
    class to class, four standard deviations of their mean."""
    n, v, d = 1 << 20, 64, 16
    g = gen(2)
    w, x = normal(g, v, d, dtype=dtype, std=0.01), (1 + 0.1 * normal(g, n, d)).to(dtype)
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    _, lse = L.linear_cross_entropy_forward(x, w, t)
    rw = torch.full((n,), 64.0 / n if dtype is torch.float16 else 1.0, device="cuda")
    _, want, _ = R.ce_backward(x, w, t, lse, rw)
    _, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, need_x=False,
                                            grad_weight=torch.empty(v, d, dtype=dtype, device="cuda"))
    mean = float(((dw[1:].double() - want[1:]) / want[1:]).mean())
    assert abs(mean) <= (128 * 4 * 4 + n / 64 / 128) * R.U + 4 * 2 ** 0.5 * R.half_step(dtype) / (3 * 63) ** 0.5
    assert off(dw[0], want[0]) <= 2 * R.half_step(dtype)


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("d", [256, 2048, 5000])
def test_logits_of_terms_of_one_sign(d, dtype):
    """Logits near 20 all of whose terms are positive.  A product of 16 cuts a sum by less than
    a step of its last place, two half steps; float16 sums end after 16 steps of four
    products, bfloat16 ones after 32; what the segments' sums, the exponentials, their sum and
    the logarithm add is what test_linear_ce_gpu allows."""
    g = gen(d)
    n, v = 300, 2000
    x = (1 + 0.3 * normal(g, n, d)).abs().to(dtype)
    w = ((1 + 0.3 * normal(g, v, d)).abs() * 20 / d).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    loss, lse = L.linear_cross_entropy_forward(x, w, t)
    want, exact, size = R.ce_forward(x, w, t, None)
    units = 2 * min(4 * (32 if dtype is torch.bfloat16 else 16), d / 16) + d / 1024 + 4
    R.within(lse, exact, 1, units * size + 300 + 4 * exact, "lse")
    R.within(loss, want, 1, units * size + 300 + 8 * exact + 4 * want, "loss")


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("n", [13, 300, 2100])
def test_the_same_bits_again_captured_and_after_anything_in_the_workspace(n, dtype):
    """16-bit gradients, and grad_x alone, with weights of 0, padding and a class most rows have."""
    v, d = 1003, 101
    x, w, t, rw = inputs(gen(n), n, v, d, dtype)
    t[::3] = 7
    rw[::5] = 0
    _, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)

    def both(x, rw):
        dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw,
                                                 grad_weight=torch.empty(v, d, dtype=dtype, device="cuda"))
        only, _ = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw, need_weight=False)
        return dx, dw, only

    want = both(x, rw)
    from learned_optimizer_step_gb300 import train_ops
    for buf, _, _ in train_ops._workspaces.values():
        buf.fill_(255)
    assert all(map(torch.equal, both(x, rw), want))
    other = rw.flip(0).contiguous()
    want_other = both(x, other)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph, buf = torch.cuda.CUDAGraph(), rw.clone()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            got = both(x, buf)
    for weights, right in ((rw, want), (other, want_other), (rw, want)):
        buf.copy_(weights)
        graph.replay()
        torch.cuda.synchronize()
        assert all(map(torch.equal, got, right))
