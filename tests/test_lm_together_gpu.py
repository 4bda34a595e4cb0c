"""The language model operators as they are used, on the GPU: a whole training step's
gradients against autograd in float64, captured and replayed, on other streams, beside
autograd."""

import math

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from examples import train_small_lm as E
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def test_example_runs():
    losses = E.main(steps=3, batch=512, show=False)
    assert len(losses) == 3 and all(map(math.isfinite, losses))


def test_gradients_of_the_example():
    """Some ten tensors between a loss and its first layer are rounded to bfloat16, each by
    2^-9 of its size at most: gradients within 10 * 2^-9 * 2 (forward and backward)."""
    model, text = E.Model(), E.Text()
    tokens, following = text.batch(700)
    loss = model.loss_and_gradients(tokens, following)
    p = {k: (model.copies[k] if k in model.copies else v).double().requires_grad_() for k, v in model.params.items()}
    norm = lambda v: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)   # noqa: E731
    x = p["table"][tokens] * E.WIDTH ** 0.5
    y0 = torch.nn.functional.layer_norm(x, (E.WIDTH,), p["n0.w"], p["n0.b"])
    s1 = x + E.SCALE * torch.sigmoid(y0 @ p["g1"]) * norm(y0 @ p["w1"]) * p["n1.post"]
    s2 = s1 + E.SCALE * norm((norm(s1) * p["n1.pre"]) @ p["w2"]) * p["n2.post"]
    z = (norm(s2) * p["n2.pre"]) @ p["head"].t()
    live = following >= 0
    want = torch.where(live, torch.logsumexp(z, 1) - z.gather(1, following.clamp(min=0)[:, None])[:, 0], 0.0)
    assert float((loss.double() - want.detach()).abs().max()) <= 10 * 2 ** -9 * float(want.detach().max())
    want.mean().backward()
    for k, g in model.grads.items():
        d = float((g.double() - p[k].grad).norm() / p[k].grad.norm())
        assert d <= 20 * 2 ** -9, (k, d)


def test_a_captured_step_replays():
    """The whole step in a graph: the same bits as eager calls, at every replay's new batch."""
    text = E.Text()
    batches = [text.batch(300) for _ in range(3)]
    eager, graphed = E.Model(), E.Model()
    tokens, following = (t.clone() for t in batches[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            loss = graphed.loss_and_gradients(tokens, following)
            norm = graphed.optimizer.step(1, 1e-3, max_norm=1.0, seed=5)
    for b in batches:
        tokens.copy_(b[0])
        following.copy_(b[1])
        graph.replay()
        want = eager.loss_and_gradients(*b)
        n = eager.optimizer.step(1, 1e-3, max_norm=1.0, seed=5)
        assert torch.equal(loss, want) and torch.equal(norm, n)
        for k in eager.params:
            assert torch.equal(eager.params[k], graphed.params[k]) and torch.equal(eager.grads[k], graphed.grads[k]), k
    L.check_indices()


def test_two_graphs_and_eager_calls_do_not_share_scratch():
    g = gen(3)
    x = [normal(g, 400, 64, dtype=torch.bfloat16) for _ in range(2)]
    w = normal(g, 900, 64, dtype=torch.bfloat16, std=0.1)
    t = torch.randint(0, 900, (400,), generator=g, device="cuda")

    def both(v):
        loss, lse = L.linear_cross_entropy_forward(v, w, t)
        return (loss, *L.linear_cross_entropy_backward(v, w, t, lse))

    want = [[r.clone() for r in both(v)] for v in x]
    graphs, outs = [], []
    for v in x:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph, stream=s):
                outs.append(both(v))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        mine = both(x[0])
        torch.cuda.synchronize()
        assert all(map(torch.equal, mine, want[0]))
        for got, right in zip(outs, want):
            assert all(map(torch.equal, got, right))


def calls():
    """Per operator: its inputs, and the call on clones of them, which gives tensors."""
    g = gen(5)
    n, cols, bf = 1024, 1024, torch.bfloat16
    h, r, gate, dy = (normal(g, n, cols, dtype=bf) for _ in range(4))
    w = normal(g, cols, mean=1.0, std=0.1)
    _, x, r1, r2 = L.block_norm_forward(h, r, w, w.clone(), gate=gate)
    table = normal(g, 2000, cols, dtype=bf, std=0.03)
    t = torch.randint(0, 2000, (n,), generator=g, device="cuda")
    _, lse = L.linear_cross_entropy_forward(h, table, t)
    p, m, v = normal(g, n * cols), normal(g, n * cols, std=1e-3), normal(g, n * cols, std=1e-3).square()

    def adamw(s, p, gr, m, v):
        norm = L.AdamW([L.AdamWTensor(p, gr, m, v)]).step(3, 1e-3, max_norm=1.0, stream=s)
        return (norm,)

    return [([h, r, w, w.clone(), gate], lambda s, h, r, a, b, q: L.block_norm_forward(h, r, a, b, gate=q, stream=s)),
            ([dy, h, x, r1, r2, w, w.clone(), gate],
             lambda s, *a: L.block_norm_backward(*a[:7], gate=a[7], stream=s)),
            ([h, table, t], lambda s, *a: L.linear_cross_entropy_forward(*a, stream=s)),
            ([h, table, t, lse], lambda s, *a: L.linear_cross_entropy_backward(*a, stream=s)),
            ([p, dy.reshape(-1), m, v], adamw)]


@pytest.mark.parametrize("k", range(5))
def test_inputs_may_be_dropped_after_a_call_on_another_stream(k):
    inputs, call = calls()[k]
    want = call(None, *[t.clone() for t in inputs])
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
    assert all(map(torch.equal, got, want))


def test_streams_of_others_and_raw_handles():
    inputs, call = calls()[2]
    want = call(None, *inputs)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream, torch.cuda.ExternalStream(s.cuda_stream)):
        got = call(stream, *inputs)
        s.synchronize()
        assert all(map(torch.equal, got, want))


@pytest.mark.parametrize("k", range(4))
def test_beside_autograd(k):
    inputs, call = calls()[k]
    floats = [t for t in inputs if t.is_floating_point() and t.dtype is not torch.float32][:2]
    versions = [t._version for t in inputs]
    call(None, *inputs)
    assert versions == [t._version for t in inputs]          # nothing of theirs is written
    for t in floats:
        t.requires_grad_()
        with pytest.raises(RuntimeError, match="not recorded by autograd"):
            call(None, *inputs)
        with torch.no_grad():
            call(None, *inputs)
        t.requires_grad_(False)


def test_written_tensors_count_as_changed():
    g = gen(1)
    x, w = normal(g, 8, 64, dtype=torch.float16), normal(g, 30, 64, dtype=torch.float16)
    t = torch.randint(0, 30, (8,), generator=g, device="cuda")
    loss, lse = (torch.zeros(8, device="cuda") for _ in range(2))
    dx, dw = torch.zeros_like(x), torch.zeros(30, 64, device="cuda")
    p = L.AdamWTensor.zeros(torch.zeros(300, device="cuda"), torch.ones(300, device="cuda"), "8bit", torch.bfloat16)
    written = (loss, lse, dx, dw, p.param, p.m, p.v, p.m_scale, p.v_scale, p.copy)
    before = [v._version for v in written]
    L.linear_cross_entropy_forward(x, w, t, loss=loss, lse=lse)
    L.linear_cross_entropy_backward(x, w, t, lse, grad_x=dx, grad_weight=dw)
    L.AdamW([p]).step(1, 0.1)
    assert all(v._version > b for v, b in zip(written, before))


def test_calls_of_several_threads():
    import threading
    inputs, call = calls()[3]
    want = [t.clone() for t in call(None, *inputs)]
    bad = []

    def work():
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                got = call(None, *inputs)
                s.synchronize()
                if not all(map(torch.equal, got, want)):
                    bad.append(1)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad
