"""Python binding of the language model operators (include/lopt_lm.h): argument
marshalling only.

Block norm and linear cross entropy are calls like the training operators'
(train_ops): on torch tensors, enqueued on ``stream`` (default: torch's current
stream), with results in the tensors given or in new ones, recorded by no
autograd; the same rules for streams, matrices and refusals hold.  AdamW is an
object that keeps a list of tensors, as LearnedOptimizer's prepared list does,
and steps it.
"""

from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch

from . import lopt as _lopt
from . import train_ops as _ops
from .lopt import load_library
from .train_ops import BF16, F16, F32, _Call, _index, _like, _matrix, _same_lead, _type, _TYPES, _vector

LM_EXPORTED = ("lopt_block_norm_forward", "lopt_block_norm_workspace", "lopt_block_norm_backward",
               "lopt_linear_ce_workspace", "lopt_linear_ce_forward", "lopt_linear_ce_backward",
               "lopt_selftest_linear_ce",
               "lopt_adamw_check", "lopt_adamw_workspace", "lopt_adamw_step", "lopt_adamw_moments")

ADAMW_BLOCK = 256


class LoptAdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("grad_type", ctypes.c_int32), ("copy_type", ctypes.c_int32),
                ("moments", ctypes.c_int32), ("decay", ctypes.c_int32)]


_fns = None


def _load():
    """The library's functions with their argument types, once."""
    global _fns
    if _fns is None:
        _ops._load()
        lib = load_library()
        vp, i32, i64, f, d = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double
        pi64, pt, pvp = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(LoptAdamWTensor), ctypes.POINTER(vp)
        sig = {
            "lopt_block_norm_forward": [vp, i32, i64, i64, i64, vp, i64, vp, i64, vp, vp, i32, f, f, vp, i64, vp, i64,
                                        vp, vp, vp],
            "lopt_block_norm_workspace": [i64, i64, pi64],
            "lopt_block_norm_backward": [vp, i32, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i32, f,
                                         vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i32, vp, i64, vp],
            "lopt_linear_ce_workspace": [i64, i64, i64, i32, i32, i32, pi64],
            "lopt_linear_ce_forward": [vp, i32, i64, i64, i64, vp, i64, i64, vp, i32, vp, vp, vp, vp, i64, vp, vp],
            "lopt_linear_ce_backward": [vp, i32, i64, i64, i64, vp, i64, i64, vp, i32, vp, vp, vp, i64, vp, i32, i64,
                                        i32, vp, i64, vp, vp],
            "lopt_adamw_check": [pt, i32],
            "lopt_adamw_workspace": [pi64],
            "lopt_adamw_step": [pt, i32, i64, d, d, d, d, d, d, ctypes.c_uint32, vp, vp, i64, vp],
            "lopt_adamw_moments": [pt, i32, pvp, pvp, vp],
        }
        sig["lopt_selftest_linear_ce"] = [i64] + sig["lopt_linear_ce_forward"]
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, i32
        _fns = {name: getattr(lib, name) for name in sig}
    return _fns


_sizes = {}


def _size_of(name, *sizes):
    """What a workspace function of the library says for these sizes."""
    need = _sizes.get((name, sizes))
    if need is None:
        got = ctypes.c_int64()
        code = _load()[name](*sizes, got)
        if code:
            _lopt._check(name, code)
        if len(_sizes) > 1024:
            _sizes.clear()
        need = _sizes[(name, sizes)] = got.value
    return need


def _run(c, name, written, *args):
    """The library's call on the device of `c`; `written`: the tensors that it writes."""
    fn = (_fns or _load())[name]
    if c.dev == _ops._current_device():
        code = fn(*args)
    else:
        with torch.cuda.device(c.dev):
            code = fn(*args)
    if code:
        _lopt._check(name, code)
    _ops._increment_version(written)


# ---- block norm -------------------------------------------------------------------


def _norm_weights(w_post, w_pre, x, cols):
    dtype = w_post.dtype
    if dtype is not torch.float32 and dtype is not x.dtype:
        raise TypeError("w_post must be float32 or of the type of h")
    return _vector(w_post, cols, "w_post", dtype), _vector(w_pre, cols, "w_pre", dtype), _TYPES[dtype]


def block_norm_forward(h, residual, w_post, w_pre, *, gate=None, scale: float = 1.0, eps: float = 1e-6, out=None,
                       summed=None, rstd_post=None, rstd_pre=None, stream=None):
    """What stands between two blocks of a language model, over the last dimension:

        summed = residual + scale * sigmoid(gate) * rmsnorm(h) * w_post
        y = rmsnorm(summed) * w_pre

    Returns (y, summed, rstd_post, rstd_pre): y goes into the next block,
    summed is what the residual stream goes on with; the two rstd (float32, one
    per row) are what the backward pass wants.  h: the block's output; gate:
    shaped like h, or None for none; w_post and w_pre: float32 or the type of h.
    ``out`` and ``summed`` may be h, residual or gate, which they then replace."""
    c = _Call(h, (residual, w_post, w_pre, gate), (out, summed, rstd_post, rstd_pre), stream)
    rows, cols, hs = _matrix(h, "h")
    if h.dim() > 2:
        _same_lead(h.shape[:-1], residual=(residual, 1), gate=(gate, 1), out=(out, 1), summed=(summed, 1),
                   rstd_post=(rstd_post, 0), rstd_pre=(rstd_pre, 0))
    kind, shape = _type(h, "h"), (rows, cols)
    w1, w2, wt = _norm_weights(w_post, w_pre, h, cols)
    if residual is None:
        raise TypeError("the operators take torch tensors")
    residual, r, rs = _like(c, residual, h, shape, "residual")
    g = gs = 0
    if gate is not None:
        gate, g, gs = _like(c, gate, h, shape, "gate")
    out, y, ys = _like(c, out, h, shape, "out")
    summed, s, ss = _like(c, summed, h, shape, "summed")
    if rstd_post is None:
        rstd_post = c.empty(h.shape[:-1], torch.float32)
    if rstd_pre is None:
        rstd_pre = c.empty(h.shape[:-1], torch.float32)
    _run(c, "lopt_block_norm_forward", (out, summed, rstd_post, rstd_pre), h.data_ptr(), kind, rows, cols, hs, r, rs, g,
         gs, w1, w2, wt, scale, eps, y, ys, s, ss, _vector(rstd_post, rows, "rstd_post"),
         _vector(rstd_pre, rows, "rstd_pre"), c.handle)
    return out, summed, rstd_post, rstd_pre


def block_norm_backward(grad_out, h, summed, rstd_post, rstd_pre, w_post, w_pre, *, gate=None, scale: float = 1.0,
                        grad_summed=None, grad_h=None, grad_residual=None, grad_gate=None, grad_w_post=None,
                        grad_w_pre=None, accumulate: bool = False, stream=None):
    """The backward pass: (grad_h, grad_residual, grad_gate or None, grad_w_post, grad_w_pre).

    grad_out: the gradient of y; grad_summed: the gradient that reaches summed
    past the norm, if any; grad_w_post and grad_w_pre: float32 [cols], the
    parameters' gradient buffers (``accumulate`` adds to them).  grad_h,
    grad_residual and grad_gate may each replace one of grad_out, h, summed,
    gate and grad_summed."""
    c = _Call(grad_out, (h, summed, w_post, w_pre, gate, grad_summed),
              (rstd_post, rstd_pre, grad_h, grad_residual, grad_gate, grad_w_post, grad_w_pre), stream)
    rows, cols, ds = _matrix(grad_out, "grad_out")
    if grad_out.dim() > 2:
        _same_lead(grad_out.shape[:-1], h=(h, 1), summed=(summed, 1), rstd_post=(rstd_post, 0),
                   rstd_pre=(rstd_pre, 0), gate=(gate, 1), grad_summed=(grad_summed, 1), grad_h=(grad_h, 1),
                   grad_residual=(grad_residual, 1), grad_gate=(grad_gate, 1))
    kind, shape = _type(grad_out, "grad_out"), (rows, cols)
    for t in (h, summed, rstd_post, rstd_pre):
        if t is None:
            raise TypeError("the operators take torch tensors")
    h, hp, hs = _like(c, h, grad_out, shape, "h")
    summed, x, xs = _like(c, summed, grad_out, shape, "summed")
    w1, w2, wt = _norm_weights(w_post, w_pre, grad_out, cols)
    g = gs = gg = ggs = s = ss = 0
    if gate is not None:
        gate, g, gs = _like(c, gate, grad_out, shape, "gate")
        grad_gate, gg, ggs = _like(c, grad_gate, grad_out, shape, "grad_gate")
    elif grad_gate is not None:
        raise ValueError("grad_gate needs a gate")
    if grad_summed is not None:
        grad_summed, s, ss = _like(c, grad_summed, grad_out, shape, "grad_summed")
    if accumulate and (grad_w_post is None or grad_w_pre is None):
        raise ValueError("accumulate needs grad_w_post and grad_w_pre")
    grad_h, gh, ghs = _like(c, grad_h, grad_out, shape, "grad_h")
    grad_residual, gr, grs = _like(c, grad_residual, grad_out, shape, "grad_residual")
    if grad_w_post is None:
        grad_w_post = c.empty((cols,), torch.float32)
    if grad_w_pre is None:
        grad_w_pre = c.empty((cols,), torch.float32)
    need = _size_of("lopt_block_norm_workspace", rows, cols)
    ws, ws_ptr = c.workspace(need)
    written = [t for t in (grad_h, grad_residual, grad_gate, grad_w_post, grad_w_pre) if t is not None]
    _run(c, "lopt_block_norm_backward", written, grad_out.data_ptr(), kind, rows, cols, ds, hp, hs, x, xs, g, gs,
         _vector(rstd_post, rows, "rstd_post"), _vector(rstd_pre, rows, "rstd_pre"), w1, w2, wt, scale, s, ss, gh, ghs,
         gr, grs, gg, ggs, _vector(grad_w_post, cols, "grad_w_post"), _vector(grad_w_pre, cols, "grad_w_pre"),
         1 if accumulate else 0, ws_ptr, need, c.handle)
    return grad_h, grad_residual, grad_gate, grad_w_post, grad_w_pre


# ---- linear cross entropy ------------------------------------------------------------


def _hidden(c, x, weight, target, row_weight):
    """What both directions say of their inputs: (type, rows, cols, x stride,
    classes, weight stride, index type, row_weight's address, rows aligned)."""
    rows, cols, xs = _matrix(x, "x")
    if x.dtype is not torch.float16 and x.dtype is not torch.bfloat16:
        raise TypeError("x must be float16 or bfloat16, not %s" % x.dtype)
    if weight.dim() != 2 or weight.shape[1] != cols:
        raise ValueError("weight must be [classes, %d]" % cols)
    if weight.dtype is not x.dtype:
        raise TypeError("weight must be of the type of x")
    classes, _, ws = _matrix(weight, "weight")
    kind = _index(target, "target")
    if target.numel() != rows:
        raise ValueError("x has %d rows for %d targets" % (rows, target.numel()))
    if x.dim() > 2:
        _same_lead(x.shape[:-1], target=(target, 0), row_weight=(row_weight, 0))
    w = 0 if row_weight is None else _vector(row_weight, rows, "row_weight")
    aligned = (x.data_ptr() % 16 == 0 and (rows <= 1 or (xs % 8 == 0 and cols <= xs < 1 << 38))
               and weight.data_ptr() % 16 == 0 and (classes <= 1 or (ws % 8 == 0 and cols <= ws < 1 << 38)))
    return _TYPES[x.dtype], rows, cols, xs, classes, ws, kind, w, 1 if aligned else 0


def linear_cross_entropy_forward(x, weight, target, *, row_weight=None, loss=None, lse=None, stream=None):
    """(loss, lse), float32, one per row: the cross entropy of the softmax of
    ``x @ weight.t()`` with each row's target, without keeping the logits.

        lse = logsumexp(x @ weight.t()),  loss = row_weight * (lse - logit of the target)

    x: [..., cols], weight: [classes, cols], both float16 or bfloat16; target:
    int32 or int64 of x's leading dimensions, negative for none (padding); a row
    without a target or with weight 0 has loss 0.  lse is what the backward pass
    wants; -(loss) with row_weight None is the target's log probability."""
    c = _Call(x, (weight, row_weight), (target, loss, lse), stream)
    kind, rows, cols, xs, classes, ws, ik, w, aligned = _hidden(c, x, weight, target, row_weight)
    if x.dim() > 2:
        _same_lead(x.shape[:-1], loss=(loss, 0), lse=(lse, 0))
    if loss is None:
        loss = c.empty(x.shape[:-1], torch.float32)
    if lse is None:
        lse = c.empty(x.shape[:-1], torch.float32)
    need = _size_of("lopt_linear_ce_workspace", rows, classes, cols, aligned, 0, F32)
    work, work_ptr = c.workspace(need)
    _run(c, "lopt_linear_ce_forward", (loss, lse), x.data_ptr(), kind, rows, cols, xs, weight.data_ptr(), classes, ws,
         target.data_ptr(), ik, w, _vector(loss, rows, "loss"), _vector(lse, rows, "lse"), work_ptr, need,
         _ops._status_ptr(c.dev), c.handle)
    return loss, lse


def linear_cross_entropy_backward(x, weight, target, lse, *, row_weight=None, grad_x=None, grad_weight=None,
                                  need_x: bool = True, need_weight: bool = True, accumulate: bool = False,
                                  stream=None):
    """(grad_x or None, grad_weight or None): the gradients of the sum of the
    rows' losses, from the forward pass's lse; row_weight is then the gradient
    that reaches each row's unweighted loss.

    grad_weight: float32 [classes, cols] (default; ``accumulate`` adds to it),
    or a buffer of the type of x, which with many tokens takes a quarter fewer
    products: what of G is not a target's is rounded to that type once.  Rows without a target or of weight 0 get zeros and add
    nothing, whatever they hold."""
    c = _Call(x, (weight, row_weight), (target, lse, grad_x, grad_weight), stream)
    kind, rows, cols, xs, classes, ws, ik, w, aligned = _hidden(c, x, weight, target, row_weight)
    if x.dim() > 2:
        _same_lead(x.shape[:-1], lse=(lse, 0), grad_x=(grad_x, 1))
    if lse is None:
        raise TypeError("the operators take torch tensors")
    if accumulate and (grad_weight is None or not need_weight):
        raise ValueError("accumulate needs grad_weight")
    gx = gxs = gw = gws = 0
    gt = kind
    written = []
    if need_x:
        grad_x, gx, gxs = _like(c, grad_x, x, (rows, cols), "grad_x")
        written.append(grad_x)
    elif grad_x is not None:
        raise ValueError("grad_x is given, need_x is not")
    if need_weight:
        if grad_weight is None:
            grad_weight = c.empty((classes, cols), torch.float32)
        gr, gc, gws = _matrix(grad_weight, "grad_weight")
        if (gr, gc) != (classes, cols):
            raise ValueError("grad_weight must be %s" % ((classes, cols),))
        if grad_weight.dtype is not torch.float32 and grad_weight.dtype is not x.dtype:
            raise TypeError("grad_weight must be float32 or of the type of x")
        gt = _TYPES[grad_weight.dtype]
        if accumulate and gt != F32:
            raise TypeError("accumulate needs a float32 grad_weight")
        gw = grad_weight.data_ptr()
        written.append(grad_weight)
    elif grad_weight is not None:
        raise ValueError("grad_weight is given, need_weight is not")
    need = _size_of("lopt_linear_ce_workspace", rows, classes, cols, aligned, 1, gt)
    work, work_ptr = c.workspace(need)
    _run(c, "lopt_linear_ce_backward", written, x.data_ptr(), kind, rows, cols, xs, weight.data_ptr(), classes, ws,
         target.data_ptr(), ik, w, _vector(lse, rows, "lse"), gx, gxs, gw, gt, gws, 1 if accumulate else 0, work_ptr,
         need, _ops._status_ptr(c.dev), c.handle)
    return (grad_x if need_x else None), (grad_weight if need_weight else None)


# ---- AdamW ------------------------------------------------------------------------


@dataclass
class AdamWTensor:
    """One parameter tensor with its gradient and moments, all contiguous and
    on one GPU.

    param: float32; grad: float32, float16 or bfloat16; m and v: float32 like
    param, or int8 and uint8 codes with m_scale and v_scale, float32, one per
    256 elements; copy: float16 or bfloat16, receives the rounded weights;
    decay: whether weight decay applies."""
    param: "object"
    grad: "object"
    m: "object"
    v: "object"
    m_scale: Optional["object"] = None
    v_scale: Optional["object"] = None
    copy: Optional["object"] = None
    decay: bool = True

    @staticmethod
    def zeros(param, grad, moments: str = "float32", copy_dtype=None, decay: bool = True) -> "AdamWTensor":
        """The state before the first step: moments ("float32" or "8bit") of
        zero, and a copy of the weights of ``copy_dtype`` if given."""
        if moments not in ("float32", "8bit"):
            raise ValueError('moments must be "float32" or "8bit"')
        n, dev = param.numel(), param.device
        copy = None if copy_dtype is None else param.detach().to(copy_dtype)
        if moments == "float32":
            m, v = (torch.zeros(n, dtype=torch.float32, device=dev) for _ in range(2))
            return AdamWTensor(param, grad, m, v, copy=copy, decay=decay)
        blocks = (n + ADAMW_BLOCK - 1) // ADAMW_BLOCK
        ms, vs = (torch.zeros(blocks, dtype=torch.float32, device=dev) for _ in range(2))
        return AdamWTensor(param, grad, torch.zeros(n, dtype=torch.int8, device=dev),
                           torch.zeros(n, dtype=torch.uint8, device=dev), ms, vs, copy, decay)

    def to_c(self) -> LoptAdamWTensor:
        def ptr(t, n, what, dtypes):
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s must be a torch.Tensor" % what)
            if not t.is_cuda or t.dtype not in dtypes or not t.is_contiguous():
                raise TypeError("%s must be a contiguous CUDA tensor of %s" % (what, " or ".join(map(str, dtypes))))
            if t.numel() != n:
                raise ValueError("%s has %d elements, expected %d" % (what, t.numel(), n))
            return t.data_ptr()

        n = self.param.numel() if isinstance(self.param, torch.Tensor) else 0
        f32, half = (torch.float32,), (torch.float16, torch.bfloat16)
        c = LoptAdamWTensor()
        c.param = ptr(self.param, n, "param", f32)
        c.grad = ptr(self.grad, n, "grad", f32 + half)
        c.grad_type = _TYPES[self.grad.dtype]
        if (self.m_scale is None) != (self.v_scale is None):
            raise ValueError("8-bit moments need m_scale and v_scale, 32-bit ones neither")
        if self.m_scale is None:
            c.m, c.v, c.moments = ptr(self.m, n, "m", f32), ptr(self.v, n, "v", f32), 32
        else:
            blocks = (n + ADAMW_BLOCK - 1) // ADAMW_BLOCK
            c.m, c.v, c.moments = ptr(self.m, n, "m", (torch.int8,)), ptr(self.v, n, "v", (torch.uint8,)), 8
            c.m_scale, c.v_scale = (ptr(t, blocks, w, f32) for t, w in ((self.m_scale, "m_scale"),
                                                                        (self.v_scale, "v_scale")))
        if self.copy is not None:
            c.copy = ptr(self.copy, n, "copy", half)
            c.copy_type = _TYPES[self.copy.dtype]
        else:
            c.copy_type = BF16
        c.n, c.decay = n, 1 if self.decay else 0
        return c


class AdamW:
    """AdamW over a list of tensors, as one call per step.

    The list is marshalled once: the tensors must stay where they are.  An
    ``AdamWTensor``'s moments are updated in place; they and the step count are
    all the state that there is."""

    def __init__(self, tensors: Sequence[AdamWTensor], *, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay: float = 0.01):
        self.tensors = list(tensors)
        if not self.tensors:
            raise ValueError("AdamW needs at least one tensor")
        self.beta1, self.beta2, self.eps, self.weight_decay = float(beta1), float(beta2), float(eps), float(weight_decay)
        self._array = (LoptAdamWTensor * len(self.tensors))(*[t.to_c() for t in self.tensors])
        self._params = [t.param for t in self.tensors]
        self._all = [x for t in self.tensors for x in (t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.copy)
                     if x is not None]
        self._written = [x for t in self.tensors for x in (t.param, t.m, t.v, t.m_scale, t.v_scale, t.copy)
                         if x is not None]
        dev = self._params[0].get_device()
        if any(x.get_device() != dev for x in self._all):
            raise TypeError("all tensors of a list must be on the same CUDA device")
        self.numel = sum(p.numel() for p in self._params)
        code = _load()["lopt_adamw_check"](self._array, len(self.tensors))
        if code:
            _lopt._check("lopt_adamw_check", code)

    def _call(self, others, stream):
        c = _Call(self._params[0], (), others, stream)
        if torch.is_grad_enabled() and any(p.requires_grad for p in self._params):
            raise RuntimeError("the step is not recorded by autograd: with parameters that require a gradient, call "
                               "it under torch.no_grad()")
        if c.stream is not None and not isinstance(c.stream, torch.cuda.ExternalStream):
            for x in self._all:
                x.record_stream(c.stream)
        return c

    def step(self, t: int, lr: float, *, max_norm: Optional[float] = None, seed: Optional[int] = None, norm=None,
             stream=None):
        """Enqueue step number ``t`` (1 for the first) and return at once.

        max_norm: clip the gradients by the norm of all of them together
        (math.inf: only look at it) and return that norm, a float32 scalar on
        the GPU (``norm``, or a new one); with a norm that is not finite the
        step changes nothing.  None: no clipping, returns None.  seed: of the
        rounding of 8-bit moments (default: t).  Captured in a graph, t, lr,
        max_norm and seed are those of the capture in every replay."""
        clipped = max_norm is not None
        if clipped and not max_norm > 0:
            raise ValueError("max_norm must be above 0")
        c = self._call((norm,) if clipped else (), stream)
        ws_ptr = need = norm_ptr = 0
        if clipped:
            need = _size_of("lopt_adamw_workspace")
            ws, ws_ptr = c.workspace(need)
            if norm is None:
                norm = c.empty((), torch.float32)
            norm_ptr = _vector(norm, 1, "norm")
        _run(c, "lopt_adamw_step", self._written + [norm] if clipped else self._written, self._array,
             len(self.tensors), int(t), float(lr), self.beta1, self.beta2, self.eps, self.weight_decay,
             float(max_norm) if clipped else 0.0, int(t if seed is None else seed) & 0xFFFFFFFF, norm_ptr, ws_ptr, need,
             c.handle)
        return norm if clipped else None

    def moments(self, m: Optional[List] = None, v: Optional[List] = None, *, stream=None):
        """The moments as float32 values, ([m of each tensor], [v of each]):
        what 8-bit codes stand for.  m and v: tensors to write into (default: new)."""
        n = len(self.tensors)
        c = self._call((*(m or ()), *(v or ())), stream)
        m, v = (list(x) if x is not None else [c.empty(p.shape, torch.float32) for p in self._params] for x in (m, v))
        if len(m) != n or len(v) != n:
            raise ValueError("one m and one v per tensor")
        arrays = [(ctypes.c_void_p * n)(*[_vector(x, p.numel(), what) for x, p in zip(xs, self._params)])
                  for xs, what in ((m, "m"), (v, "v"))]
        _run(c, "lopt_adamw_moments", m + v, self._array, n, *arrays, c.handle)
        return m, v
