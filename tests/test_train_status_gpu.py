"""Reports of bad indices on the GPU, each in a process of its own, since what
matters is the first call: captured, in inference mode, or by several threads
at once."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import threading
import torch
import learned_optimizer_step_gb300 as L
from learned_optimizer_step_gb300 import train_ops as ops
table, index = torch.ones(10, 16, device="cuda"), torch.tensor([3, 10, -1, 9], device="cuda")
z, t = torch.zeros(300, 9001, device="cuda"), torch.zeros(300, 3, device="cuda")
i = torch.zeros(300, 3, dtype=torch.int64, device="cuda")
torch.cuda.synchronize()

def reported():
    try:
        L.check_indices()
    except L.LoptError as e:
        assert e.code == ops.E_INDEX, e
        return True
    return False
"""

FIRST_CALL_CAPTURED = """
def capture(f):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        keep = f()
    return graph, keep
lookup = capture(lambda: L.embedding_forward(table, index))
loss = capture(lambda: L.distill_forward_backward(z, t, i))
back = capture(lambda: L.embedding_backward(table[:4], index, 10))
assert not reported()                    # nothing has run
lookup[0].replay()
assert reported() and not reported()
assert lookup[1][:, 0].tolist() == [1, 0, 0, 1]
loss[0].replay()
assert not reported()
i[7, 1] = 9001
loss[0].replay()
assert reported()
back[0].replay()
assert reported() and not reported()
lookup[0].replay(), lookup[0].replay()
assert reported() and not reported()
"""

FIRST_CALL_IN_INFERENCE_MODE = """
with torch.inference_mode():
    L.embedding_forward(table, index)
assert reported() and not reported()
L.embedding_forward(table, index)
with torch.inference_mode():
    assert reported() and not reported()
"""

FIRST_CALLS_OF_THREADS = """
gate, got = threading.Barrier(8), []

def first():
    gate.wait()
    got.append(ops._status_ptr(0))
threads = [threading.Thread(target=first) for _ in range(8)]
[x.start() for x in threads], [x.join() for x in threads]
assert len(got) == 8 and len(set(got)) == 1 and got[0], got

def call():
    gate.wait()
    for _ in range(50):
        L.embedding_forward(table, index)
for _ in range(3):
    threads = [threading.Thread(target=call) for _ in range(8)]
    [x.start() for x in threads], [x.join() for x in threads]
    assert reported() and not reported()
"""


@pytest.mark.parametrize("body", [FIRST_CALL_CAPTURED, FIRST_CALL_IN_INFERENCE_MODE, FIRST_CALLS_OF_THREADS],
                         ids=["captured", "inference mode", "threads"])
def test_first_call(body):
    need_gpu()
    r = subprocess.run([sys.executable, "-c", HEAD + body], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
