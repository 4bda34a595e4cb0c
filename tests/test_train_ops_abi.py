"""CPU checks of the training operators' C ABI (include/lopt_train.h): the
exports, and every refusal that needs no device.  Only calls that must be
refused are made, with addresses that are never read."""

import ctypes
import math
import os
import re

import pytest

from learned_optimizer_step_gb300 import build as B

torch = pytest.importorskip("torch")

from learned_optimizer_step_gb300 import lopt as L   # noqa: E402
from learned_optimizer_step_gb300 import train_ops as ops   # noqa: E402

HEADER = os.path.join(B.ROOT, "include", "lopt_train.h")
ARG, SHAPE, ALIGN, ALIAS = -1, -2, -3, -8
F32, F16, BF16, I32, I64 = 0, 1, 2, 0, 1


@pytest.fixture(scope="module")
def fns():
    B.build()
    return ops._load()


def test_exports_are_the_header(fns):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lopt_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(ops.TRAIN_EXPORTED) == sorted(fns)
    values = dict(re.findall(r"#define (LOPT_\w+)\s+(-?\d+)", open(HEADER).read()))
    assert (int(values["LOPT_F32"]), int(values["LOPT_F16"]), int(values["LOPT_BF16"])) == (ops.F32, ops.F16, ops.BF16)
    assert int(values["LOPT_E_INDEX"]) == ops.E_INDEX and int(values["LOPT_MAX_TOP"]) == ops.MAX_TOP
    assert L.load_library().lopt_strerror(ops.E_INDEX).decode() == "index out of range"


def test_package_names():
    import learned_optimizer_step_gb300 as pkg
    assert pkg.embedding_forward is ops.embedding_forward and pkg.distill_forward is ops.distill_forward
    with pytest.raises(AttributeError):
        pkg.no_such_operator


# One accepted-looking call of each function, by argument name, and changes
# that must be refused.  The addresses are apart from each other: 1 << 40 on.
MB = 1 << 20
A = [(1 << 40) + k * 64 * MB for k in range(16)]

FWD = dict(table=A[0], table_type=F32, rows=100, cols=64, table_stride=64, index=A[1], index_type=I64, n=10, scale=1.0,
           out=A[2], out_type=BF16, out_stride=64, status=A[3], stream=0)
BWD = dict(grad_out=A[0], type=BF16, grad_out_stride=64, index=A[1], index_type=I32, n=10, rows=100, cols=64, scale=1.0,
           accumulate=0, grad=A[2], workspace=A[4], workspace_bytes=MB, status=0, stream=0)
NF = dict(x=A[0], type=F16, rows=10, cols=64, x_stride=64, residual=A[1], residual_stride=64, weight=A[2], bias=A[3],
          weight_type=F32, eps=1e-5, y=A[4], y_stride=64, summed=A[5], summed_stride=64, mean=A[6], rstd=A[7], stream=0)
NB = dict(grad_out=A[0], type=F32, rows=10, cols=64, grad_out_stride=64, x=A[1], x_stride=64, mean=A[2], rstd=A[3],
          weight=A[4], weight_type=F32, grad_residual=A[5], grad_residual_stride=64, grad_x=A[6], grad_x_stride=64,
          grad_weight=A[7], grad_bias=A[8], accumulate=0, workspace=A[9], workspace_bytes=MB, stream=0)
KD = dict(logits=A[0], type=BF16, rows=10, cols=64, logits_stride=64, top_logits=A[1], top_type=F32,
          top_logits_stride=8, top_index=A[2], index_type=I64, top_index_stride=8, top=8, temperature=1.0,
          row_weight=A[3], loss=A[4], grad=A[5], grad_stride=64, status=A[6], stream=0)

REFUSED = [
    ("lopt_embed_forward", FWD, [
        (dict(table=0), ARG), (dict(index=0), ARG), (dict(out=0), ARG), (dict(table_type=3), ARG),
        (dict(out_type=-1), ARG), (dict(index_type=2), ARG), (dict(rows=0), SHAPE), (dict(cols=0), SHAPE),
        (dict(n=-1), SHAPE), (dict(n=1 << 31), SHAPE), (dict(cols=(1 << 23) + 1), SHAPE), (dict(table_stride=-1), SHAPE),
        (dict(out_stride=63), SHAPE), (dict(table=A[0] + 2), ALIGN), (dict(out=A[2] + 1), ALIGN),
        (dict(index=A[1] + 4), ALIGN), (dict(status=A[3] + 2), ALIGN), (dict(out=A[0]), ALIAS),
        (dict(out=A[0] + 128), ALIAS), (dict(out=A[1]), ALIAS)]),
    ("lopt_embed_backward", BWD, [
        (dict(grad_out=0), ARG), (dict(grad=0), ARG), (dict(workspace=0), ARG), (dict(workspace_bytes=16), ARG),
        (dict(type=9), ARG), (dict(accumulate=2), ARG), (dict(rows=0), SHAPE), (dict(n=-1), SHAPE),
        (dict(grad=A[2] + 2), ALIGN), (dict(workspace=A[4] + 16), ALIGN), (dict(grad_out=A[0] + 1), ALIGN),
        (dict(grad_out_stride=-64), SHAPE), (dict(grad=A[0]), ALIAS), (dict(workspace=A[2]), ALIAS),
        (dict(workspace=A[0]), ALIAS), (dict(grad=A[1]), ALIAS)]),
    ("lopt_layernorm_forward", NF, [
        (dict(x=0), ARG), (dict(weight=0), ARG), (dict(y=0), ARG), (dict(mean=0), ARG), (dict(rstd=0), ARG),
        (dict(type=5), ARG), (dict(weight_type=BF16), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG),
        (dict(residual=0), ARG), (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(y_stride=0), SHAPE),
        (dict(x=A[0] + 1), ALIGN), (dict(bias=A[3] + 2), ALIGN), (dict(mean=A[6] + 2), ALIGN),
        (dict(y=A[0] + 128), ALIAS), (dict(y=A[0], y_stride=128), ALIAS), (dict(y=A[5]), ALIAS),
        (dict(rstd=A[6] + 8), ALIAS), (dict(mean=A[2]), ALIAS), (dict(y=A[3]), ALIAS), (dict(mean=A[0]), ALIAS)]),
    ("lopt_layernorm_backward", NB, [
        (dict(grad_out=0), ARG), (dict(x=0), ARG), (dict(grad_x=0), ARG), (dict(grad_weight=0), ARG),
        (dict(mean=0), ARG), (dict(workspace=0), ARG), (dict(workspace_bytes=8), ARG), (dict(accumulate=-1), ARG),
        (dict(weight_type=F16), ARG), (dict(cols=0), SHAPE), (dict(grad_x_stride=8), SHAPE),
        (dict(grad_weight=A[7] + 2), ALIGN), (dict(workspace=A[9] + 128), ALIGN), (dict(grad_bias=A[7]), ALIAS),
        (dict(grad_x=A[0] + 256), ALIAS), (dict(grad_weight=A[4]), ALIAS), (dict(workspace=A[6]), ALIAS),
        (dict(grad_x=A[2]), ALIAS), (dict(grad_bias=A[1] + 64), ALIAS)]),
    ("lopt_distill", KD, [
        (dict(logits=0), ARG), (dict(top_logits=0), ARG), (dict(top_index=0), ARG), (dict(loss=0), ARG),
        (dict(type=3), ARG), (dict(top_type=F16), ARG), (dict(index_type=-1), ARG), (dict(temperature=0.0), ARG),
        (dict(temperature=-1.0), ARG), (dict(temperature=math.nan), ARG), (dict(temperature=math.inf), ARG),
        (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(top=0), SHAPE), (dict(top=1025), SHAPE),
        (dict(grad_stride=63), SHAPE), (dict(logits=A[0] + 1), ALIGN), (dict(grad=A[5] + 1), ALIGN),
        (dict(row_weight=A[3] + 2), ALIGN), (dict(status=A[6] + 1), ALIGN), (dict(grad=A[0] + 64), ALIAS),
        (dict(grad=A[0], grad_stride=65), ALIAS), (dict(loss=A[5]), ALIAS), (dict(loss=A[0]), ALIAS),
        (dict(loss=A[3]), ALIAS), (dict(grad=A[1]), ALIAS), (dict(grad=A[2]), ALIAS)]),
]


@pytest.mark.parametrize("name,base,changes", REFUSED, ids=[r[0] for r in REFUSED])
def test_refusals(fns, name, base, changes):
    for change, code in changes:
        assert fns[name](*{**base, **change}.values()) == code, (name, change)


def test_nothing_to_do_is_no_launch(fns):
    assert fns["lopt_embed_forward"](*{**FWD, "n": 0}.values()) == 0
    assert fns["lopt_embed_backward"](*{**BWD, "n": 0, "accumulate": 1}.values()) == 0
    assert fns["lopt_layernorm_forward"](*{**NF, "rows": 0}.values()) == 0
    assert fns["lopt_layernorm_backward"](*{**NB, "rows": 0, "accumulate": 1}.values()) == 0
    assert fns["lopt_distill"](*{**KD, "rows": 0}.values()) == 0


def test_workspace_sizes(fns):
    need = ctypes.c_int64()
    for n, rows, cols in ((0, 1, 1), (1, 1, 1), (4099, 50257, 768), (65536, 50304, 2048), (1 << 30, 1 << 30, 64)):
        assert fns["lopt_embed_workspace"](n, rows, cols, need) == 0
        assert need.value >= 8 * n + 4 * (rows + 1)      # positions, ids, first positions
    assert fns["lopt_embed_workspace"](-1, 1, 1, need) == SHAPE
    assert fns["lopt_embed_workspace"](1, 1, 1, None) == ARG
    for rows, cols in ((0, 1), (1, 1), (32768, 2048), (1 << 30, 1 << 20)):
        assert fns["lopt_layernorm_workspace"](rows, cols, need) == 0
        assert need.value >= 8 * cols and need.value % 4 == 0
    assert fns["lopt_layernorm_workspace"](1, 0, need) == SHAPE
    assert fns["lopt_layernorm_workspace"](1, 1, None) == ARG


def test_binding_refuses_cpu_tensors():
    t, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: ops.embedding_forward(t, i), lambda: ops.embedding_backward(t, i, 4),
                 lambda: ops.layernorm_forward(t, t[0]), lambda: ops.distill_forward(t, t, i),
                 lambda: ops.layernorm_backward(t, t, t[:, 0], t[:, 0], t[0])):
        with pytest.raises(TypeError):
            call()
