"""CPU checks of the language model operators' C ABI (include/lopt_lm.h): the exports,
the struct, the workspaces, and every refusal that needs no device.  Only calls that
must be refused are made, with addresses that are never read."""

import ctypes
import math
import os
import random
import re

import pytest

from learned_optimizer_step_gb300 import build as B

torch = pytest.importorskip("torch")

from learned_optimizer_step_gb300 import lm_ops as ops   # noqa: E402

HEADER = os.path.join(B.ROOT, "include", "lopt_lm.h")
ARG, SHAPE, ALIGN, ALIAS = -1, -2, -3, -8
F32, F16, BF16, I32, I64 = 0, 1, 2, 0, 1


@pytest.fixture(scope="module")
def fns():
    B.build()
    return ops._load()


def test_exports_are_the_header(fns):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lopt_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(ops.LM_EXPORTED) == sorted(fns)
    assert int(re.search(r"#define LOPT_ADAMW_BLOCK (\d+)", open(HEADER).read()).group(1)) == ops.ADAMW_BLOCK


def test_struct_layout():
    # seven pointers, an int64 and four int32, natural alignment, no padding
    assert ctypes.sizeof(ops.LoptAdamWTensor) == 7 * 8 + 8 + 4 * 4
    assert ops.LoptAdamWTensor.n.offset == 56 and ops.LoptAdamWTensor.decay.offset == 76


def test_package_names():
    import learned_optimizer_step_gb300 as pkg
    assert pkg.AdamW is ops.AdamW and pkg.block_norm_forward is ops.block_norm_forward
    assert pkg.linear_cross_entropy_backward is ops.linear_cross_entropy_backward


MB = 1 << 20
A = [(1 << 40) + k * 64 * MB for k in range(20)]

NF = dict(h=A[0], type=BF16, rows=10, cols=64, h_stride=64, residual=A[1], residual_stride=64, gate=A[2], gate_stride=64,
          w_post=A[3], w_pre=A[4], weight_type=F32, scale=1.0, eps=1e-6, y=A[5], y_stride=64, summed=A[6], summed_stride=64,
          rstd_post=A[7], rstd_pre=A[8], stream=0)
NB = dict(grad_y=A[0], type=F16, rows=10, cols=64, grad_y_stride=64, h=A[1], h_stride=64, summed=A[2], summed_stride=64,
          gate=A[3], gate_stride=64, rstd_post=A[4], rstd_pre=A[5], w_post=A[6], w_pre=A[7], weight_type=F16, scale=1.0,
          grad_summed=A[8], grad_summed_stride=64, grad_h=A[9], grad_h_stride=64, grad_residual=A[10],
          grad_residual_stride=64, grad_gate=A[11], grad_gate_stride=64, grad_w_post=A[12], grad_w_pre=A[13], accumulate=0,
          workspace=A[14], workspace_bytes=MB, stream=0)
CF = dict(x=A[0], type=BF16, rows=10, cols=64, x_stride=64, weight=A[1], classes=100, weight_stride=64, target=A[2],
          index_type=I64, row_weight=A[3], loss=A[4], lse=A[5], workspace=A[6], workspace_bytes=32 * MB, status=A[7], stream=0)
CB = dict(x=A[0], type=F16, rows=10, cols=64, x_stride=64, weight=A[1], classes=100, weight_stride=64, target=A[2],
          index_type=I32, row_weight=A[3], lse=A[4], grad_x=A[5], grad_x_stride=64, grad_weight=A[6], grad_weight_type=F32,
          grad_weight_stride=64, accumulate=0, workspace=A[7], workspace_bytes=32 * MB, status=A[8], stream=0)

REFUSED = [
    ("lopt_block_norm_forward", NF, [
        (dict(h=0), ARG), (dict(residual=0), ARG), (dict(w_post=0), ARG), (dict(w_pre=0), ARG), (dict(y=0), ARG),
        (dict(summed=0), ARG), (dict(rstd_post=0), ARG), (dict(rstd_pre=0), ARG), (dict(type=3), ARG),
        (dict(weight_type=F16), ARG), (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(scale=math.inf), ARG),
        (dict(scale=math.nan), ARG), (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(rows=1 << 31), SHAPE),
        (dict(y_stride=63), SHAPE), (dict(h_stride=-1), SHAPE), (dict(h=A[0] + 1), ALIGN), (dict(gate=A[2] + 1), ALIGN),
        (dict(w_pre=A[4] + 2), ALIGN), (dict(rstd_pre=A[8] + 1), ALIGN), (dict(y=A[0] + 64), ALIAS),
        (dict(y=A[0], y_stride=128), ALIAS), (dict(summed=A[5]), ALIAS), (dict(y=A[3]), ALIAS), (dict(rstd_post=A[8]), ALIAS),
        (dict(rstd_post=A[0]), ALIAS), (dict(summed=A[4]), ALIAS)]),
    ("lopt_block_norm_backward", NB, [
        (dict(grad_y=0), ARG), (dict(h=0), ARG), (dict(summed=0), ARG), (dict(gate=0), ARG), (dict(grad_gate=0), ARG),
        (dict(grad_h=0), ARG), (dict(grad_residual=0), ARG), (dict(grad_w_post=0), ARG), (dict(grad_w_pre=0), ARG),
        (dict(workspace=0), ARG), (dict(workspace_bytes=8), ARG), (dict(accumulate=2), ARG), (dict(weight_type=BF16), ARG),
        (dict(scale=math.nan), ARG), (dict(cols=0), SHAPE), (dict(grad_h_stride=8), SHAPE), (dict(workspace=A[14] + 128), ALIGN),
        (dict(grad_w_pre=A[13] + 2), ALIGN), (dict(grad_h=A[10]), ALIAS), (dict(grad_h=A[1] + 128), ALIAS),
        (dict(grad_w_post=A[13]), ALIAS), (dict(grad_w_post=A[6]), ALIAS), (dict(workspace=A[4]), ALIAS),
        (dict(grad_gate=A[9]), ALIAS), (dict(grad_residual=A[5]), ALIAS)]),
    ("lopt_linear_ce_forward", CF, [
        (dict(x=0), ARG), (dict(weight=0), ARG), (dict(target=0), ARG), (dict(loss=0), ARG), (dict(lse=0), ARG),
        (dict(workspace=0), ARG), (dict(workspace_bytes=64), ARG), (dict(type=F32), ARG), (dict(type=7), ARG),
        (dict(index_type=2), ARG), (dict(rows=-1), SHAPE), (dict(rows=(1 << 22) + 1), SHAPE), (dict(classes=0), SHAPE),
        (dict(classes=(1 << 22) + 1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=(1 << 16) + 1), SHAPE),
        (dict(x_stride=-64), SHAPE), (dict(x=A[0] + 1), ALIGN), (dict(target=A[2] + 4), ALIGN), (dict(row_weight=A[3] + 2), ALIGN),
        (dict(lse=A[5] + 1), ALIGN), (dict(status=A[7] + 1), ALIGN), (dict(workspace=A[6] + 128), ALIGN), (dict(loss=A[5]), ALIAS),
        (dict(loss=A[0]), ALIAS), (dict(lse=A[3]), ALIAS), (dict(workspace=A[1]), ALIAS), (dict(loss=A[2]), ALIAS)]),
    ("lopt_linear_ce_backward", CB, [
        (dict(x=0), ARG), (dict(weight=0), ARG), (dict(target=0), ARG), (dict(lse=0), ARG), (dict(workspace=0), ARG),
        (dict(workspace_bytes=64), ARG), (dict(type=F32), ARG), (dict(accumulate=3), ARG), (dict(grad_weight_type=BF16), ARG),
        (dict(grad_weight_type=F16, accumulate=1), ARG), (dict(classes=0), SHAPE), (dict(grad_x_stride=63), SHAPE),
        (dict(grad_weight_stride=63), SHAPE), (dict(grad_weight=A[6] + 2), ALIGN), (dict(grad_x=A[5] + 1), ALIGN),
        (dict(lse=A[4] + 2), ALIGN), (dict(grad_x=A[0]), ALIAS), (dict(grad_weight=A[1]), ALIAS), (dict(grad_x=A[6]), ALIAS),
        (dict(grad_x=A[4]), ALIAS), (dict(workspace=A[6]), ALIAS), (dict(grad_weight=A[3]), ALIAS)]),
]


@pytest.mark.parametrize("name,base,changes", REFUSED, ids=[r[0] for r in REFUSED])
def test_refusals(fns, name, base, changes):
    for change, code in changes:
        assert fns[name](*{**base, **change}.values()) == code, (name, change)


def test_the_self_test_refuses_what_the_call_does(fns):
    for limit in (-1, 10 ** 9 + 1):
        assert fns["lopt_selftest_linear_ce"](limit, *CF.values()) == ARG
    for change, code in REFUSED[2][2]:
        assert fns["lopt_selftest_linear_ce"](0, *{**CF, **change}.values()) == code, change


def test_nothing_to_do_is_no_launch(fns):
    assert fns["lopt_block_norm_forward"](*{**NF, "rows": 0}.values()) == 0
    assert fns["lopt_block_norm_backward"](*{**NB, "rows": 0, "accumulate": 1}.values()) == 0
    assert fns["lopt_linear_ce_forward"](*{**CF, "rows": 0}.values()) == 0
    assert fns["lopt_linear_ce_backward"](*{**CB, "rows": 0, "accumulate": 1}.values()) == 0
    assert fns["lopt_linear_ce_backward"](*{**CB, "grad_x": 0, "grad_weight": 0}.values()) == 0
    assert fns["lopt_adamw_step"](None, 0, 1, 0.1, 0.9, 0.999, 1e-8, 0.0, 0.0, 1, None, None, 0, None) == 0


def test_workspace_sizes(fns):
    need = ctypes.c_int64()
    ce = fns["lopt_linear_ce_workspace"]
    for rows, classes, cols in ((0, 1, 1), (1, 1, 1), (7, 50257, 768), (8192, 50304, 2048), (1 << 22, 1 << 22, 8)):
        assert ce(rows, classes, cols, 1, 0, F32, need) == 0
        plain = need.value
        assert ce(rows, classes, cols, 0, 0, F32, need) == 0 and need.value >= plain + 2 * classes * cols
        assert ce(rows, classes, cols, 1, 1, BF16, need) == 0
        half = need.value
        assert half >= 6 * rows * cols          # x, and grad_x in fp32
        assert ce(rows, classes, cols, 1, 1, F32, need) == 0 and need.value >= half
    # G of a chunk stays within half a gigabyte while 256 classes of it do.
    assert ce(8192, 50304, 2048, 1, 1, F32, need) == 0 and need.value < 800 * MB
    for bad, code in (((-1, 1, 1, 1, 0, F32), SHAPE), ((1, 0, 1, 1, 0, F32), SHAPE), ((1, 1, 1, 2, 0, F32), ARG),
                      ((1, 1, 1, 1, 5, F32), ARG), ((1, 1, 1, 1, 1, 9), ARG)):
        assert ce(*bad, need) == code
    assert ce(1, 1, 1, 1, 0, F32, None) == ARG
    for rows, cols in ((0, 1), (1, 1), (32768, 2048), (1 << 30, 1 << 20)):
        assert fns["lopt_block_norm_workspace"](rows, cols, need) == 0 and need.value >= 8 * cols + 4 * rows
    assert fns["lopt_block_norm_workspace"](1, 0, need) == SHAPE and fns["lopt_block_norm_workspace"](1, 1, None) == ARG
    assert fns["lopt_adamw_workspace"](need) == 0 and need.value > 0 and fns["lopt_adamw_workspace"](None) == ARG


def test_the_size_asked_for_is_enough(fns):
    """Over the range of sizes, with either gradient left out.  The calls stop at a
    workspace that is not aligned, which is looked at after its size."""
    rng, need = random.Random(7), ctypes.c_int64()
    spread = lambda low, high: int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))   # noqa: E731
    sizes = [(4099, 50257, 128), (4099, 50257, 64), (12000, 16384, 128), (19000, 8000, 64), (6000, 50257, 128), (256, 1 << 20, 8)]
    sizes += [(spread(1, 60000), spread(1, 200000), spread(1, 3000)) for _ in range(4000)]
    far = [(k + 1) << 50 for k in range(8)]
    for rows, classes, cols in sizes:
        cols8 = (cols + 7) // 8 * 8
        for dtype in (F16, BF16):
            for asked, given in ((F32, F32), (dtype, dtype), (F32, None), (dtype, None)):
                assert fns["lopt_linear_ce_workspace"](rows, classes, cols, 1, 1, asked, need) == 0
                call = {**CB, "type": dtype, "rows": rows, "cols": cols, "x_stride": cols8, "classes": classes, "weight_stride": cols8,
                        "grad_x_stride": cols, "grad_weight": 0 if given is None else far[0], "grad_weight_stride": cols,
                        "grad_weight_type": asked, "x": far[1], "weight": far[2], "target": far[3], "row_weight": far[4],
                        "lse": far[5], "grad_x": far[6], "workspace": far[7] + 128, "workspace_bytes": need.value}
                code = fns["lopt_linear_ce_backward"](*call.values())
                assert code == ALIGN, (rows, classes, cols, dtype, asked, given, code)
        assert fns["lopt_linear_ce_workspace"](rows, classes, cols, 1, 0, F32, need) == 0
        call = {**CF, "rows": rows, "cols": cols, "x_stride": cols8, "classes": classes, "weight_stride": cols8, "x": far[1],
                "weight": far[2], "target": far[3], "row_weight": far[4], "loss": far[5], "lse": far[6], "workspace": far[7] + 128,
                "workspace_bytes": need.value}
        assert fns["lopt_linear_ce_forward"](*call.values()) == ALIGN


def tensor(**change):
    t = ops.LoptAdamWTensor()
    for k, v in {**dict(param=A[0], grad=A[1], m=A[2], v=A[3], n=1000, grad_type=F32, copy_type=BF16, moments=32, decay=1),
                 **change}.items():
        setattr(t, k, v)
    return t


def test_adamw_refusals(fns):
    ok = dict(n=1, t=1, lr=0.1, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, max_norm=0.0, seed=1, norm=None,
              workspace=None, workspace_bytes=0, stream=None)
    step = lambda tensor_, **k: fns["lopt_adamw_step"]((ops.LoptAdamWTensor * 1)(tensor_), *{**ok, **k}.values())   # noqa: E731
    for change, code in ((dict(param=0), ARG), (dict(grad=0), ARG), (dict(m=0), ARG), (dict(v=0), ARG), (dict(n=-1), SHAPE),
                         (dict(n=(1 << 40) + 1), SHAPE), (dict(grad_type=5), ARG), (dict(moments=16), ARG), (dict(decay=2), ARG),
                         (dict(moments=8), ARG), (dict(copy=A[4], copy_type=F32), ARG), (dict(param=A[0] + 2), ALIGN),
                         (dict(grad=A[1] + 1, grad_type=F16), ALIGN), (dict(copy=A[4] + 1), ALIGN), (dict(m=A[0]), ALIAS),
                         (dict(v=A[2] + 400), ALIAS), (dict(grad=A[3]), ALIAS), (dict(copy=A[1]), ALIAS),
                         (dict(moments=8, m_scale=A[5], v_scale=A[5]), ALIAS)):
        assert step(tensor(**change)) == code, change
        assert fns["lopt_adamw_check"]((ops.LoptAdamWTensor * 1)(tensor(**change)), 1) == code, change
    for change in (dict(t=0), dict(lr=math.nan), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(eps=-1.0),
                   dict(eps=math.inf), dict(weight_decay=math.nan), dict(max_norm=-1.0), dict(max_norm=math.nan), dict(n=-1),
                   dict(max_norm=1.0), dict(max_norm=1.0, norm=A[8]), dict(max_norm=1.0, norm=A[8], workspace=A[9], workspace_bytes=8)):
        assert step(tensor(), **change) == ARG, change
    big = dict(max_norm=1.0, norm=A[8], workspace=A[9], workspace_bytes=MB)
    assert step(tensor(), **{**big, "workspace": A[9] + 16}) == ALIGN
    assert step(tensor(), **{**big, "norm": A[0]}) == ALIAS and step(tensor(), **{**big, "workspace": A[2]}) == ALIAS
    assert step(tensor(), **{**big, "norm": A[9] + 64}) == ALIAS
    two = lambda a, b: fns["lopt_adamw_check"]((ops.LoptAdamWTensor * 2)(a, b), 2)   # noqa: E731
    other = dict(param=A[5], grad=A[6], m=A[7], v=A[8])
    assert two(tensor(), tensor(**other)) == 0
    assert two(tensor(), tensor(**{**other, "grad": A[1] + 400})) == 0       # gradients may overlap
    assert two(tensor(), tensor(**{**other, "grad": A[0]})) == ALIAS
    assert two(tensor(), tensor(**{**other, "m": A[3] + 4})) == ALIAS
    assert two(tensor(), tensor(**{**other, "param": A[1] + 4})) == ALIAS


def test_binding_refuses_cpu_tensors():
    t, i = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    for call in (lambda: ops.block_norm_forward(t, t, t[0], t[0]), lambda: ops.linear_cross_entropy_forward(t, t, i),
                 lambda: ops.block_norm_backward(t, t, t, f, f, t[0], t[0]),
                 lambda: ops.linear_cross_entropy_backward(t, t, i, f),
                 lambda: ops.AdamW([ops.AdamWTensor(f, f, f, f)]), lambda: ops.AdamW([ops.AdamWTensor(None, f, f, f)])):
        with pytest.raises(TypeError):
            call()
