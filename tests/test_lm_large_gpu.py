"""The language model operators on tensors whose offsets pass 31 and 32 bits, on the
GPU: their far ends against the references."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from tests import lm_reference as R
from tests.gpu_helpers import need_gpu
from tests.test_block_norm_gpu import check_backward, check_forward
from tests.test_train_ops_gpu import gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    yield
    L.release_workspaces()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_a_table_of_more_than_2_to_31_elements(kind):
    n, v, d = 6, 1_100_003, 2048
    g = gen(1)
    w = torch.empty(v, d, dtype=torch.bfloat16, device="cuda").normal_(0, d ** -0.5, generator=g)
    x = normal(g, n, d, dtype=torch.bfloat16)
    t = torch.tensor([0, v - 1, v - 1, 1_048_576, 555_555, -1], device="cuda")
    loss, lse = L.linear_cross_entropy_forward(x, w, t)
    z = torch.cat([x.double() @ w[k:k + 100_000].double().t() for k in range(0, v, 100_000)], 1)
    want = torch.logsumexp(z, 1)
    assert float((lse.double() - want).abs().max()) <= 2e-5
    chosen = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    assert float((loss.double() - torch.where(t >= 0, want - chosen, 0.0)).abs().max()) <= 4e-5
    dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, grad_weight=torch.empty(v, d, dtype=kind, device="cuda"))
    p = torch.exp(z - lse.double()[:, None])
    p[torch.arange(n, device="cuda"), t.clamp(min=0)] -= 1
    p[5] = 0
    for rows in (slice(0, 300), slice(1_048_500, 1_048_700), slice(v - 300, v)):
        want = p[:, rows].t() @ x.double()
        assert float((dw[rows].double() - want).norm()) <= (2e-5 if kind is torch.float32 else 2 ** -7) * float(want.norm())
    want = sum(p[:, k:k + 100_000] @ w[k:k + 100_000].double() for k in range(0, v, 100_000))
    assert float((dx.double() - want).norm()) <= 2 ** -7 * float(want.norm())


def test_more_than_2_to_22_over_tiles_of_tokens():
    """300,000 tokens: several forward launches, chunks of 256 classes."""
    n, v, d = 300_000, 700, 24
    g = gen(2)
    x, w = normal(g, n, d, dtype=torch.float16), normal(g, v, d, dtype=torch.float16, std=0.3)
    t = torch.randint(-1, v, (n,), generator=g, device="cuda")
    rw = torch.rand(n, generator=g, device="cuda")
    loss, lse = L.linear_cross_entropy_forward(x, w, t, row_weight=rw)
    want, wl, size = R.ce_forward(x, w, t, rw)
    assert float((lse.double() - wl).abs().max()) <= 1e-5 and float((loss.double() - want).abs().max()) <= 2e-5
    dx, dw = L.linear_cross_entropy_backward(x, w, t, lse, row_weight=rw)
    rx, rd, _ = R.ce_backward(x, w, t, lse, rw)
    assert float((dw.double() - rd).norm()) <= 1e-5 * float(rd.norm())
    assert float((dx.double() - rx).norm()) <= 2 ** -10 * float(rx.norm())


def test_adamw_past_32_bits():
    n = (1 << 32) + 70_001
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t = L.AdamWTensor(p, g, torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda"),
                      *[torch.zeros((n + 255) // 256, device="cuda") for _ in range(2)])
    rng = np.random.default_rng(1)
    places = [slice(0, 1024), slice((1 << 31) - 512, (1 << 31) + 512), slice((1 << 32) - 512, (1 << 32) + 512), slice(n - 70_001 + 1024 * 60, n)]
    data = []
    for s in places:
        k = s.stop - s.start
        p[s] = torch.from_numpy(rng.normal(size=k).astype(np.float32)).cuda()
        g[s] = torch.from_numpy(rng.normal(size=k).astype(np.float32) * np.float32(0.01)).cuda().bfloat16()
        data.append((p[s].cpu().numpy(), g[s].float().cpu().numpy()))
    total = math.sqrt(sum(float((d[1].astype(np.float64) ** 2).sum()) for d in data))
    norm = L.AdamW([t]).step(1, 1e-3, max_norm=math.inf, seed=9)
    assert abs(float(norm) - total) <= total * 2.0 ** -23
    key = R.mix(np.uint64(9) ^ np.uint64(0x9E3779B9))
    for s, (p0, g0) in zip(places, data):
        zero = np.zeros(len(p0), np.float32)
        want, m, root, _ = R.adamw(p0, g0, zero, zero, 1, 1e-3, 0.9, 0.999, 1e-8, 0.01, True)
        assert np.array_equal(p[s].cpu().numpy(), want), s
        i = np.arange(s.start, s.stop, dtype=np.uint64)
        bits = R.mix((i & np.uint64(0xFFFFFFFF)) ^ key ^ ((i >> np.uint64(32)) * np.uint64(0x85EBCA6B) & np.uint64(0xFFFFFFFF)))
        assert np.array_equal(t.m[s].cpu().numpy().astype(np.int64), R.encode(m, 127, bits >> np.uint64(16))[0]), s
        assert np.array_equal(t.v[s].cpu().numpy().astype(np.int64), R.encode(root, 255, bits & np.uint64(0xFFFF))[0]), s


def test_block_norm_past_31_bits():
    rows, cols = 262_200, 8200
    g = gen(3)
    h, r, dy = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(3))
    w1, w2 = normal(g, cols, mean=1.0, std=0.1), normal(g, cols, mean=1.0, std=0.1)
    got = L.block_norm_forward(h, r, w1, w2, scale=0.5)
    for s in (slice(0, 5), slice(rows - 5, rows)):
        check_forward([t[s] for t in got], h[s], r[s], w1, w2, None, 0.5)
    back = L.block_norm_backward(dy, h, *got[1:], w1, w2, scale=0.5)
    for s in (slice(0, 5), slice(rows - 5, rows)):
        x, a, b = (t[s] for t in got[1:])
        want, size = R.norm_backward(dy[s], h[s], x, a, b, w1, w2, None, 0.5, None)
        for k in (0, 1):
            R.within(back[k][s], want[k], 3 * 189, size[k])
