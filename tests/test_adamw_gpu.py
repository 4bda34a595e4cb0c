"""AdamW on the GPU: bit for bit against float32 arithmetic done operation by operation
(numpy), near the definition in 64 bits, with ragged and unaligned tensors, 8-bit
moments, clipping, and what it refuses."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from learned_optimizer_step_gb300 import LoptError
from tests import lm_reference as R
from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
H = dict(lr=3e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.1)


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def make(rng, n, eight, grad=torch.float32, copy=None, decay=True, shift=0, std=1e-2):
    """A tensor and its numpy originals; `shift` elements off the allocation's alignment."""
    def dev(a, dtype):
        buf = torch.zeros(len(a) + shift + 64, dtype=dtype, device="cuda")
        t = buf[shift:shift + len(a)]
        t.copy_(torch.as_tensor(a))
        return t
    p = rng.normal(size=n).astype(np.float32)
    g = dev(rng.normal(size=n) * std, grad)
    blocks = -(-n // 256)
    if eight:
        o = dict(m=rng.integers(-127, 128, n).astype(np.int8), v=rng.integers(0, 256, n).astype(np.uint8),
                 ms=(rng.random(blocks) * 1e-6).astype(np.float32), vs=(rng.random(blocks) * 1e-6).astype(np.float32))
        t = L.AdamWTensor(dev(p, torch.float32), g, dev(o["m"], torch.int8), dev(o["v"], torch.uint8),
                          dev(o["ms"], torch.float32), dev(o["vs"], torch.float32))
        o["m32"], o["v32"] = R.decode(o["m"], o["ms"], False), R.decode(o["v"], o["vs"], True)
    else:
        o = dict(m32=(rng.normal(size=n) * std).astype(np.float32), v32=((rng.normal(size=n) * std) ** 2).astype(np.float32))
        t = L.AdamWTensor(dev(p, torch.float32), g, dev(o["m32"], torch.float32), dev(o["v32"], torch.float32))
    t.copy = None if copy is None else dev(p, copy)
    t.decay = decay
    o.update(p=p, g=g.float().cpu().numpy(), n=n)
    return t, o


def check(t, o, index, step, seed, clip=np.float32(1)):
    p, m, root, v = R.adamw(o["p"], o["g"], o["m32"], o["v32"], step, H["lr"], H["b1"], H["b2"], H["eps"], H["wd"], t.decay, clip)
    assert np.array_equal(t.param.cpu().numpy(), p)
    if t.copy is not None:
        assert torch.equal(t.copy.cpu(), torch.from_numpy(p).to(t.copy.dtype))
    if t.m_scale is None:
        assert np.array_equal(t.m.cpu().numpy(), m) and np.array_equal(t.v.cpu().numpy(), v)
        return
    key = R.mix(np.uint64(seed) ^ np.uint64((index + 1) * 0x9E3779B9 & 0xFFFFFFFF))
    bits = R.mix(np.arange(o["n"], dtype=np.uint64) ^ key)
    for codes, scale, x, top, b in ((t.m, t.m_scale, m, 127, bits >> np.uint64(16)), (t.v, t.v_scale, root, 255, bits & np.uint64(0xFFFF))):
        want, s = R.encode(x, top, b)
        assert np.array_equal(scale.cpu().numpy(), s)
        assert np.array_equal(codes.cpu().numpy().astype(np.int64), want)


def opt(tensors):
    return L.AdamW(tensors, beta1=H["b1"], beta2=H["b2"], eps=H["eps"], weight_decay=H["wd"])


GRADS = [torch.float32, torch.float16, torch.bfloat16]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("n", [1, 3, 255, 256, 257, 1000, 2047, 2048, 2049, 100003])
def test_one_tensor(n, eight):
    rng = np.random.default_rng(n)
    t, o = make(rng, n, eight, GRADS[n % 3], [None, torch.float16, torch.bfloat16][n % 3], n % 2 == 0)
    assert opt([t]).step(7, H["lr"], seed=12345) is None
    check(t, o, 0, 7, 12345)


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_unaligned(shift):
    rng = np.random.default_rng(shift)
    ts = [make(rng, 1000 + k, bool(k % 2), GRADS[k % 3], torch.bfloat16, shift=shift) for k in range(4)]
    opt([t for t, _ in ts]).step(1, H["lr"])
    for k, (t, o) in enumerate(ts):
        check(t, o, k, 1, 1)


def test_long_mixed_lists():
    """More tensors than one launch takes, of all kinds, empty ones among them."""
    rng = np.random.default_rng(5)
    ts = [make(rng, int(rng.integers(0, 3000)), bool(rng.integers(2)), GRADS[k % 3], [None, torch.float16, torch.bfloat16][k % 3],
               bool(k % 2)) for k in range(900)]
    opt([t for t, _ in ts]).step(3, H["lr"], seed=2 ** 32 - 1)
    for k, (t, o) in enumerate(ts):
        check(t, o, k, 3, 2 ** 32 - 1)


def test_large_tensor():
    rng = np.random.default_rng(6)
    ts = [make(rng, 12_000_037, eight, copy=torch.bfloat16) for eight in (False, True)]
    opt([t for t, _ in ts]).step(1000, H["lr"])
    for k, (t, o) in enumerate(ts):
        check(t, o, k, 1000, 1000)


@pytest.mark.parametrize("max_norm", [0.5, 1e6, math.inf])
def test_clipping(max_norm):
    rng = np.random.default_rng(9)
    ts = [make(rng, n, bool(n % 2), GRADS[n % 3]) for n in (5, 1000, 4096, 300001)]
    norm = opt([t for t, _ in ts]).step(2, H["lr"], max_norm=max_norm)
    want = math.sqrt(math.fsum(float(x) ** 2 for _, o in ts for x in o["g"]))
    # The squares' sum is right to some 2^-45, so that the norm is the rounded one but
    # where that hangs on less than 2^-21 of a step.
    assert abs(float(norm) - want) <= want * 2.0 ** -24 * 1.0001
    clip = np.float32(min(1.0, max_norm / (want + 1e-6)))
    for k, (t, o) in enumerate(ts):
        check(t, o, k, 2, 2, clip)


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e19, 1e30])
def test_norm_of_squares_that_leave_the_range(size):
    g = torch.full((5000,), size, device="cuda")
    g[::7] = 0
    t = L.AdamWTensor.zeros(torch.zeros(5000, device="cuda"), g)
    norm = L.AdamW([t]).step(1, 0.0, max_norm=math.inf)
    want = float(g.double().norm())
    assert abs(float(norm) - want) <= want * 2.0 ** -23


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_changes_nothing(bad):
    rng = np.random.default_rng(3)
    ts = [make(rng, 3000, eight, copy=torch.bfloat16) for eight in (False, True)]
    ts[1][0].grad[2999] = bad
    before = [[x.clone() for x in (t.param, t.m, t.v, t.copy)] for t, _ in ts]
    norm = opt([t for t, _ in ts]).step(1, H["lr"], max_norm=1.0)
    assert not math.isfinite(float(norm))
    for (t, _), b in zip(ts, before):
        assert all(map(torch.equal, (t.param, t.m, t.v, t.copy), b))


def test_against_the_definition():
    """Ten steps beside the formulas in 64 bits.  A step's rounding errors: m and v 3 half
    steps each, the root and quotient some 8, times lr; the parameter two more."""
    rng = np.random.default_rng(11)
    t, o = make(rng, 5000, False, copy=torch.float16)
    p, m, v = (o[k].astype(np.float64) for k in ("p", "m32", "v32"))
    a = opt([t])
    for k in range(1, 11):
        g = rng.normal(size=5000).astype(np.float32) * np.float32(1e-2)
        t.grad.copy_(torch.from_numpy(g))
        a.step(k, H["lr"])
        p, m, v = R.adamw_exact(p, g, m, v, k, H["lr"], H["b1"], H["b2"], H["eps"], H["wd"], True)
    got = t.param.double().cpu().numpy()
    assert np.all(np.abs(got - p) <= R.U * 10 * (3 * np.abs(p) + 40 * H["lr"] * 12))
    assert np.all(np.abs(t.v.double().cpu().numpy() - v) <= 4 * 10 * R.U * v)


def test_rounding_keeps_the_mean():
    """8-bit moments that change by less than a code's distance: over many seeds the
    decoded mean is the exact value.  Each value is one of two neighbours, at most
    (2 * 254 + 1) / 255^2 of the largest apart, so that the mean of N is off by less than
    5 * 0.5 * 0.0079 / sqrt(N) (five standard deviations)."""
    n, seeds = 256, 400
    rng = np.random.default_rng(1)
    v0 = (rng.random(n) ** 2 * 1e-4).astype(np.float32)
    v0[0] = 1.2e-4                          # the block's largest, which sets the scale
    total_m, total_r = np.zeros(n), np.zeros(n)
    m0 = (rng.normal(size=n) * 1e-3).astype(np.float32)
    m0[1] = 5e-3
    zeros = np.zeros(n, np.uint64)
    mc, ms = R.encode(m0, 127, zeros)
    vc, vs = R.encode(np.sqrt(v0), 255, zeros)
    g = (rng.normal(size=n) * 1e-3).astype(np.float32)
    _, m, root, _ = R.adamw(m0 * 0, g, R.decode(mc, ms, False), R.decode(vc, vs, True), 1, 0.0, 0.9, 0.999, 1e-8, 0.0, False)
    for seed in range(seeds):
        t = L.AdamWTensor(torch.zeros(n, device="cuda"), torch.from_numpy(g).cuda(), torch.from_numpy(mc.astype(np.int8)).cuda(),
                          torch.from_numpy(vc.astype(np.uint8)).cuda(), torch.from_numpy(ms).cuda(), torch.from_numpy(vs).cuda())
        a = L.AdamW([t])
        a.step(1, 0.0, seed=seed)
        ms_, vs_ = a.moments()
        total_m += ms_[0].double().cpu().numpy()
        total_r += vs_[0].double().sqrt().cpu().numpy()
    gap = lambda top: 2.5 * (2 * top - 1) / top ** 2 / math.sqrt(seeds)   # noqa: E731
    assert np.all(np.abs(total_m / seeds - m) <= gap(127) * np.abs(m).max())
    assert np.all(np.abs(total_r / seeds - root) <= gap(255) * root.max())


def test_moments():
    rng = np.random.default_rng(2)
    ts = [make(rng, n, eight, shift=s) for n, eight, s in ((1000, True, 0), (257, True, 1), (600, False, 0), (0, True, 0))]
    m, v = opt([t for t, _ in ts]).moments()
    for (t, o), a, b in zip(ts, m, v):
        assert np.array_equal(a.cpu().numpy().ravel(), o["m32"]) and np.array_equal(b.cpu().numpy().ravel(), o["v32"])
    t = L.AdamWTensor.zeros(torch.ones(3, 100, device="cuda"), torch.ones(3, 100, device="cuda"), "8bit", torch.bfloat16)
    a = L.AdamW([t])
    assert a.moments()[0][0].shape == (3, 100) and not bool(a.moments()[1][0].any())
    a.step(1, 0.1)
    # From zeros: m = 0.1 g, root = sqrt(0.001) |g|, the same for all, hence the largest code.
    assert bool((t.m == 127).all()) and bool((t.v == 255).all())
    assert torch.allclose(t.param, torch.full((3, 100), 0.9 - 0.001, device="cuda"), atol=1e-5)
    assert torch.equal(t.copy, t.param.bfloat16())


def test_tensors_without_elements():
    e = lambda: torch.zeros(0, device="cuda")   # noqa: E731
    a = L.AdamW([L.AdamWTensor(e(), e(), e(), e())])
    assert float(a.step(1, 0.1, max_norm=1.0)) == 0.0 and a.step(2, 0.1) is None
    assert a.moments()[0][0].shape == (0,)


def test_tiny_blocks_become_zeros():
    n = 512
    t = L.AdamWTensor.zeros(torch.zeros(n, device="cuda"), torch.full((n,), 1e-31, device="cuda"), "8bit")
    t.grad[300:] = 1e-3
    L.AdamW([t]).step(1, 1e-3)
    assert not bool(t.m[:256].any()) and not bool(t.v[:256].any()) and bool((t.m[300:] != 0).all())
    assert not bool(t.m[256:300].any())


def test_refusals():
    one = lambda n=64, **k: L.AdamWTensor.zeros(torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), **k)   # noqa: E731
    t = one()
    for change, error in ((dict(param=t.param.half()), TypeError), (dict(grad=t.grad.double()), TypeError),
                          (dict(grad=t.grad[:32]), ValueError), (dict(m=t.m.cpu()), TypeError), (dict(m=t.param), LoptError),
                          (dict(v=t.m), LoptError), (dict(copy=t.param.clone()), TypeError), (dict(m_scale=t.m[:1]), ValueError),
                          (dict(grad=t.param), LoptError), (dict(param=None), TypeError)):
        u = L.AdamWTensor(t.param, t.grad, t.m, t.v)
        for k, x in change.items():
            setattr(u, k, x)
        with pytest.raises(error):
            L.AdamW([u])
    with pytest.raises(ValueError):
        L.AdamW([])
    with pytest.raises(LoptError):          # two tensors of the list overlap
        L.AdamW([one(), t, L.AdamWTensor(t.param[32:], t.grad[32:].clone(), *[torch.zeros(32, device="cuda") for _ in range(2)])])
    shared = one()                          # gradients may be shared
    L.AdamW([t, L.AdamWTensor(shared.param, t.grad, shared.m, shared.v)]).step(1, 0.1)
    a = L.AdamW([t])
    for bad in (dict(t=0), dict(lr=math.nan), dict(lr=math.inf), dict(max_norm=-1.0), dict(max_norm=0.0), dict(max_norm=math.nan)):
        with pytest.raises((ValueError, LoptError)):
            a.step(**{**dict(t=1, lr=0.1), **bad})
    for bad in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(eps=math.nan), dict(weight_decay=math.inf)):
        with pytest.raises(LoptError):
            L.AdamW([t], **bad).step(1, 0.1)
    t.param.requires_grad_()
    with pytest.raises(RuntimeError, match="not recorded"):
        a.step(1, 0.1)
    with torch.no_grad():
        a.step(1, 0.1)
    with pytest.raises(ValueError):
        with torch.no_grad():
            a.moments([t.m], [])
