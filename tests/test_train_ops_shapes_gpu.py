"""Leading dimensions of the training operators' tensors on the GPU: flat or
alike, and refused where the same number of rows stands in another order."""

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import distill_inputs, gen, norm_inputs, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def cases():
    """(call, tensors by name that go with its first one, all of leading dimensions 2 x 3)."""
    g = gen(1)
    x, w, b = norm_inputs(g, 6, 16, torch.float32, torch.float32)
    x = x.view(2, 3, 16)
    mat = lambda: normal(g, 2, 3, 16)                       # noqa: E731
    vec = lambda: torch.ones(2, 3, device="cuda")           # noqa: E731
    index = torch.randint(0, 9, (2, 3), generator=g, device="cuda")
    z, t, i = (a.view(2, 3, -1) for a in distill_inputs(g, 6, 16, 4, torch.float32, torch.float32, torch.int64))
    table = normal(g, 9, 16)
    return [
        (lambda **k: L.embedding_forward(table, index, **k), dict(out=mat())),
        (lambda grad_out: L.embedding_backward(grad_out, index, 9), dict(grad_out=mat())),
        (lambda **k: L.layernorm_forward(x, w, b, **k),
         dict(residual=mat(), out=mat(), summed=mat(), mean=vec(), rstd=vec())),
        (lambda **k: L.layernorm_backward(mat(), weight=w, **k),
         dict(x=x, mean=vec(), rstd=vec(), grad_residual=mat(), grad_x=mat())),
        (lambda **k: L.distill_forward_backward(z, **k),
         dict(top_logits=t, top_index=i, row_weight=vec(), loss=vec(), grad=mat())),
    ]


def flat(t):
    return t.reshape(6) if t.dim() == 2 else t.reshape(6, t.shape[-1])


def other(t):
    return t.reshape(3, 2) if t.dim() == 2 else t.reshape(3, 2, t.shape[-1])


@pytest.mark.parametrize("k", range(5))
def test_leading_dimensions(k):
    call, tensors = cases()[k]
    call(**tensors)
    call(**{name: flat(t) for name, t in tensors.items()})
    for name, t in tensors.items():
        call(**{**tensors, name: flat(t)})
        call(**{**tensors, name: t.unsqueeze(0)})
        with pytest.raises(ValueError):
            call(**{**tensors, name: other(t)})


def test_the_tables_gradient_has_the_tables_shape():
    dy, index = torch.ones(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for out in (torch.zeros(5, 8, device="cuda"), torch.zeros(40, device="cuda")):
        assert float(L.embedding_backward(dy, index, 5, out=out).sum()) == 32
    for shape in ((8, 5), (10, 4), (1, 5, 8)):
        with pytest.raises(ValueError):
            L.embedding_backward(dy, index, 5, out=torch.zeros(*shape, device="cuda"))


def test_out_and_out_dtype_agree():
    table, index = torch.ones(5, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    out = torch.empty(4, 8, dtype=torch.bfloat16, device="cuda")
    L.embedding_forward(table, index, out=out, out_dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        L.embedding_forward(table, index, out=out, out_dtype=torch.float32)
