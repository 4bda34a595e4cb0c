"""The language model operators' first calls of a process, captured in a graph: nothing
has been loaded or looked up before.  In processes of their own."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = """
import torch
import learned_optimizer_step_gb300 as L
g = torch.Generator(device="cuda")
g.manual_seed(1)
n = lambda *s: torch.randn(*s, generator=g, device="cuda")
x, w = n(600, 64).bfloat16(), n(900, 64).bfloat16()
t = torch.randint(0, 900, (600,), generator=g, device="cuda")
h, r, a = n(600, 64), n(600, 64), torch.ones(64, device="cuda")
p, gr, m, v = n(5000), n(5000), n(5000), n(5000).square()


def call():
%s

s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
graph = torch.cuda.CUDAGraph()
keep = [q.clone() for q in (p, m, v)]
torch.cuda.synchronize()
with torch.cuda.stream(s):
    with torch.cuda.graph(graph, stream=s):
        got = call()
graph.replay()
torch.cuda.synchronize()
got = [q.clone() for q in got]
for q, k in zip((p, m, v), keep):
    q.copy_(k)
want = call()
torch.cuda.synchronize()
assert all(map(torch.equal, got, want))
print("fine")
"""

CALLS = {
    "linear_ce": """
    loss, lse = L.linear_cross_entropy_forward(x, w, t)
    return [loss, lse, *L.linear_cross_entropy_backward(x, w, t, lse)]
""",
    "block_norm": """
    y, q, b, c = L.block_norm_forward(h, r, a, a.clone(), gate=r)
    return [y, q, b, c, *L.block_norm_backward(y, h, q, b, c, a, a.clone(), gate=r)]
""",
    "adamw": """
    norm = L.AdamW([L.AdamWTensor(p, gr, m, v)]).step(1, 1e-3, max_norm=1.0)
    return [norm, p, m, v]
""",
}


@pytest.mark.parametrize("name", CALLS)
def test_the_first_call_may_be_captured(name):
    need_gpu()
    r = subprocess.run([sys.executable, "-c", COMMON % CALLS[name]], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr
