"""The training operators on a stream other than the current one, on the GPU:
the caller may drop the call's tensors at once."""

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import distill_inputs, gen, norm_inputs, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def operators():
    """Per operator: its inputs, and the call on clones of them."""
    g = gen(5)
    n, cols = 1024, 1024                     # tensors of 4 MB, with blocks of the allocator of their own
    x, w, b = norm_inputs(g, n, cols, torch.float32, torch.float32)
    _, mean, rstd = L.layernorm_forward(x, w, b)
    dy = normal(g, n, cols)
    index = torch.randint(0, n, (n,), generator=g, device="cuda")
    z, t, i = distill_inputs(g, n, cols, 512, torch.float32, torch.float32, torch.int64)
    return [([x, index], lambda s, x, index: L.embedding_forward(x, index, stream=s)),
            ([dy, index], lambda s, dy, index: L.embedding_backward(dy, index, n, stream=s)),
            ([x, w, b, dy], lambda s, x, w, b, r: L.layernorm_forward(x, w, b, residual=r, stream=s)),
            ([dy, x, mean, rstd, w], lambda s, *a: L.layernorm_backward(*a, stream=s)),
            ([z, t, i], lambda s, *a: L.distill_forward_backward(*a, stream=s))]


@pytest.mark.parametrize("k", range(5))
def test_inputs_may_be_dropped_after_the_call(k):
    inputs, call = operators()[k]
    want = call(None, *inputs)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    clones = [t.clone() for t in inputs]
    shapes = [(t.shape, t.dtype) for t in clones]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)        # some 20 ms: the call comes after what follows here
    got = call(s, *clones)
    del clones
    again = [torch.full(shape, 3, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(2)]
    torch.cuda.synchronize()
    del again
    same = lambda a, c: torch.equal(a, c) if a is not None else c is None   # noqa: E731
    assert all(map(same, got, want)) if isinstance(got, tuple) else same(got, want)


def test_streams_of_others_are_taken():
    table, index = torch.ones(10, 16, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream, torch.cuda.ExternalStream(s.cuda_stream)):
        out = L.embedding_forward(table, index, stream=stream)
        s.synchronize()
        assert bool((out == 1).all())
