"""Distillation under masks of every size on the GPU: classes masked by a
finite value between -1e4 and the type's lowest, at the front, at the end or
over the whole row, at several temperatures and in every kernel."""

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import check_distill, gen, ids, normal

pytestmark = pytest.mark.gpu

MASKS = {torch.float32: (-1e4, -1e7, -1e10, -1e20, -1e30, torch.finfo(torch.float32).min),
         torch.bfloat16: (-1e4, -1e10, -1e30, torch.finfo(torch.bfloat16).min),
         torch.float16: (-1e4, torch.finfo(torch.float16).min)}


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


# Rows of a warp (a slot of the list in each lane, and lists in shared memory),
# of a block, of one and of several persistent blocks, and beyond those.
@pytest.mark.parametrize("dtype", list(MASKS), ids=ids)
@pytest.mark.parametrize("cols,top", [(40, 6), (1000, 20), (999, 60), (3001, 6), (9001, 40), (50257, 6), (950003, 40)])
def test_finite_masks(dtype, cols, top):
    g = gen(cols + top)
    temperatures = (1.0, 2.0, 5.0, 8.0, 20.0) if cols < 60000 else (1.0, 8.0)
    masks = MASKS[dtype]
    rows = 3 * len(masks)
    z = normal(g, rows, cols, dtype=dtype, std=2.0)
    kept = torch.zeros(rows, cols, dtype=torch.bool, device="cuda")
    for k, mask in enumerate(masks):
        z[3 * k, :cols - cols // 4] = mask       # the front: a thread's first classes, all of most threads
        kept[3 * k, cols - cols // 4:] = True
        z[3 * k + 1, cols // 4:] = mask          # the end
        kept[3 * k + 1, :cols // 4] = True
        z[3 * k + 2] = mask                      # nothing but masked: all classes alike
        kept[3 * k + 2] = True
    draw = torch.where(kept, torch.rand(rows, cols, generator=g, device="cuda"), -1.0)
    index = torch.topk(draw, top, 1)[1]
    t = normal(g, rows, top)
    for T in temperatures:
        loss, grad = L.distill_forward_backward(z, t, index, T)
        assert torch.isfinite(loss).all() and torch.isfinite(grad).all(), T
        check_distill(z, t, index, T, None, loss, grad, "T=%g" % T)
        assert torch.equal(loss, L.distill_forward(z, t, index, T)), T


def test_logits_far_from_zero():
    """Rows whose spread is small against their distance from zero: the
    exponent may lose nothing that the logits still hold."""
    g = gen(3)
    index = torch.randint(0, 5003, (6, 8), generator=g, device="cuda")
    t = normal(g, 6, 8)
    for far in (1e5, -1e6, 3e7, -1e10):
        z = (normal(g, 6, 5003, std=2.0) + far).float()
        for T in (1.0, 8.0):
            check_distill(z, t, index, T, None, *L.distill_forward_backward(z, t, index, T), "%g, T=%g" % (far, T))
