"""The training operators' C entries after cudaDeviceReset(), which ends the
process's own context, on the GPU: the calls of a plain C program, in a process
of its own (torch does not outlive its context)."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import ctypes
import numpy as np
from learned_optimizer_step_gb300 import train_ops as ops   # its import of torch loads the runtime, and makes no context
rt = ctypes.CDLL("libcudart.so.13")
rt.cudaMalloc.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
rt.cudaMemcpy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
fns = ops._load()


def device(a):
    p = ctypes.c_void_p()
    assert rt.cudaMalloc(ctypes.byref(p), a.nbytes) == 0
    assert rt.cudaMemcpy(p, a.ctypes.data, a.nbytes, 1) == 0
    return p.value


def host(p, a):
    assert rt.cudaDeviceSynchronize() == 0
    assert rt.cudaMemcpy(a.ctypes.data, p, a.nbytes, 2) == 0
    return a


def everything(rows=100, cols=50257, n=9000):
    z = np.random.default_rng(1).standard_normal((rows, cols)).astype(np.float32)
    top, index = np.zeros((rows, 1), np.float32), np.arange(rows, dtype=np.int64)[:, None]
    dz, dt, di, dl = device(z), device(top), device(index), device(np.zeros(rows, np.float32))
    code = fns["lopt_distill"](dz, 0, rows, cols, cols, dt, 0, 1, di, 1, 1, 1, 1.0, None, dl, None, 0, None, None)
    assert code == 0, code                        # its blocks take more than 48 KB of shared memory
    want = np.log(np.exp(z.astype(np.float64)).sum(1)) - z[np.arange(rows), np.arange(rows)]
    assert np.abs(host(dl, np.zeros(rows, np.float32)) - want).max() < 1e-4
    dy, ids = np.ones((n, 16), np.float32), (np.arange(n) % 7).astype(np.int64)
    need = ctypes.c_int64()
    assert fns["lopt_embed_workspace"](n, 100000, 16, need) == 0
    dd, dn, dg, dw = device(dy), device(ids), device(np.zeros((100000, 16), np.float32)), device(np.zeros(need.value, np.int8))
    code = fns["lopt_embed_backward"](dd, 0, 16, dn, 1, n, 100000, 16, 1.0, 0, dg, dw, need.value, None, None)
    assert code == 0, code
    got = host(dg, np.zeros((100000, 16), np.float32))
    assert (got[:7, 0] == np.bincount(ids)).all() and not got[7:].any()
    word, flags = ctypes.c_void_p(), ctypes.c_int32(9)
    assert fns["lopt_status_word"](word) == 0 and word.value
    assert fns["lopt_status_take"](flags) == 0 and flags.value == 0


everything()
for _ in range(2):
    assert rt.cudaDeviceReset() == 0
    everything()
"""


def test_calls_after_a_reset():
    need_gpu()
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
