"""The training operators' scratch memory on the GPU: kept by a thread that
calls, given back when it ends or on request."""

import threading

import pytest

torch = pytest.importorskip("torch")

import learned_optimizer_step_gb300 as L
from tests import train_reference as R
from tests.gpu_helpers import need_gpu
from tests.test_train_ops_gpu import gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def inputs(n=4096, rows=300, cols=512):
    g = gen(n)
    index = torch.randint(0, rows, (n,), generator=g, device="cuda")
    dy, out = normal(g, n, cols), torch.empty(rows, cols, device="cuda")
    return dy, index, rows, out


def test_scratch_goes_with_its_thread():
    dy, index, rows, out = inputs()
    want, bound = R.embed_backward(dy, index, rows, 1.0)
    L.release_workspaces()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()

    def work():
        L.embedding_backward(dy, index, rows, out=out)
        L.embedding_backward(dy, index, rows, out=out)
    for _ in range(5):
        thread = threading.Thread(target=work)
        thread.start()
        thread.join()
        assert torch.cuda.memory_allocated() == before
    R.check(out, want, bound, "from a thread")


def test_release_reaches_every_thread():
    dy, index, rows, out = inputs()
    L.release_workspaces()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    called, go = threading.Barrier(4), threading.Event()
    outs = [torch.empty_like(out) for _ in range(3)]
    before = torch.cuda.memory_allocated()

    def work(k):
        L.embedding_backward(dy, index, rows, out=outs[k])
        called.wait()
        go.wait()
        L.embedding_backward(dy, index, rows, out=outs[k])
    threads = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    [t.start() for t in threads]
    called.wait()
    assert torch.cuda.memory_allocated() > before          # each has its own
    L.release_workspaces()
    assert torch.cuda.memory_allocated() == before
    go.set()
    [t.join() for t in threads]
    want, bound = R.embed_backward(dy, index, rows, 1.0)
    for o in outs:
        R.check(o, want, bound, "threads")
