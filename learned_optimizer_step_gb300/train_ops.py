"""Python binding of the training operators (include/lopt_train.h): argument
marshalling only.

The learned optimizer's step reads one contiguous float32 gradient per
parameter; these operators make some of them.  Each call enqueues its kernels
on ``stream`` (default: torch's current stream) and returns at once.  Results
go into the tensors given (``out=``, ``grad=`` ...: a training loop's own
gradient buffers) or into new ones.  Matrices have contiguous rows; leading
dimensions are flattened; the distance between rows is free.  There is no
fallback: a tensor that is not on the GPU, or a shape that does not fit,
raises.

With a ``stream`` other than the current one, the call does not wait for work
of the current one, and new results belong to ``stream``.  Its tensors may be
dropped at once if ``stream`` is one of torch's own; with a raw handle or an
ExternalStream the caller keeps them until that stream is done with them.

The operators record nothing for autograd: the backward passes are calls of
their own.  With gradients enabled, a tensor that requires one is refused; call
under torch.no_grad() or from a torch.autograd.Function.  Tensors that are
written count as changed in place, so that autograd notices if it had saved
them.

Indices: a negative one stands for none (padding, an unused slot).  One at or
above the limit is treated the same and reported by ``check_indices()``, since
only the device sees it.
"""

from __future__ import annotations

import ctypes
import functools
import threading
import weakref
from typing import Optional

import torch

from . import lopt as _lopt
from .lopt import LoptError, load_library

F32, F16, BF16 = 0, 1, 2
I32, I64 = 0, 1
MAX_TOP = 1024
E_INDEX = -10
_lopt.ERRORS.setdefault(E_INDEX, "LOPT_E_INDEX")

TRAIN_EXPORTED = ("lopt_embed_forward", "lopt_embed_workspace", "lopt_embed_backward", "lopt_layernorm_forward",
                  "lopt_layernorm_workspace", "lopt_layernorm_backward", "lopt_distill", "lopt_selftest_distill",
                  "lopt_status_word", "lopt_status_take")

_TYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_INDEX = {torch.int32: I32, torch.int64: I64}
_E_TIMEOUT = -7

_increment_version = torch._C._increment_version
_is_grad_enabled = torch.is_grad_enabled
_raw_stream = torch._C._cuda_getCurrentRawStream
_is_capturing = torch._C._cuda_isCurrentStreamCapturing
_current_device = torch._C._cuda_getDevice
_fns = None


def _load():
    """The library's functions with their argument types, once."""
    global _fns
    if _fns is None:
        lib = load_library()
        vp, i32, i64, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        pi64 = ctypes.POINTER(ctypes.c_int64)
        sig = {
            "lopt_embed_forward": [vp, i32, i64, i64, i64, vp, i32, i64, f, vp, i32, i64, vp, vp],
            "lopt_embed_workspace": [i64, i64, i64, pi64],
            "lopt_embed_backward": [vp, i32, i64, vp, i32, i64, i64, i64, f, i32, vp, vp, i64, vp, vp],
            "lopt_layernorm_forward": [vp, i32, i64, i64, i64, vp, i64, vp, vp, i32, f, vp, i64, vp, i64, vp, vp, vp],
            "lopt_layernorm_workspace": [i64, i64, pi64],
            "lopt_layernorm_backward": [vp, i32, i64, i64, i64, vp, i64, vp, vp, vp, i32, vp, i64, vp, i64, vp, vp,
                                        i32, vp, i64, vp],
            "lopt_distill": [vp, i32, i64, i64, i64, vp, i32, i64, vp, i32, i64, i64, f, vp, vp, vp, i64, vp, vp],
        }
        sig["lopt_status_word"] = [ctypes.POINTER(vp)]
        sig["lopt_status_take"] = [ctypes.POINTER(ctypes.c_int32)]
        sig["lopt_selftest_distill"] = [i64] + sig["lopt_distill"]
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, i32
        _fns = {name: getattr(lib, name) for name in sig}
    return _fns


# ---- tensors ------------------------------------------------------------------


def _matrix(t, what):
    """(rows, cols, row stride) of a tensor with its leading dimensions flattened."""
    shape = t.shape
    if len(shape) == 2:
        rows, cols = shape
        if t.is_contiguous():
            return rows, cols, cols
        rs, cs = t.stride()
    elif not shape:
        raise ValueError("%s must have at least one dimension" % what)
    else:
        cols = shape[-1]
        rows = t.numel() // cols if cols else 0
        try:
            rs, cs = t.view(rows, cols).stride()
        except RuntimeError:
            raise ValueError("the leading dimensions of %s cannot be flattened without a copy" % what) from None
    if cs != 1 and cols > 1:
        raise ValueError("the rows of %s must be contiguous" % what)
    return rows, cols, rs


def _type(t, what):
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise TypeError("%s must be float32, float16 or bfloat16, not %s" % (what, t.dtype)) from None


def _vector(t, n, what, dtype=torch.float32):
    """Address of a contiguous vector of n elements."""
    if t.dtype is not dtype or not t.is_contiguous():
        raise TypeError("%s must be a contiguous %s tensor" % (what, dtype))
    if t.numel() != n:
        raise ValueError("%s has %d elements, expected %d" % (what, t.numel(), n))
    return t.data_ptr()


def _index(t, what):
    try:
        kind = _INDEX[t.dtype]
    except KeyError:
        raise TypeError("%s must be int32 or int64, not %s" % (what, t.dtype)) from None
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return kind


_DEVICES = "all tensors of a call must be on the same CUDA device"


def _same_lead(lead, **tensors):
    """Tensors that are not flat have the leading dimensions of the one they go with."""
    want = [d for d in lead if d != 1]
    if len(want) < 2:
        return
    for what, (t, tail) in tensors.items():
        if t is not None and t.dim() - tail > 1 and [d for d in t.shape[:t.dim() - tail] if d != 1] != want:
            raise ValueError("%s is %s, expected leading dimensions %s" % (what, tuple(t.shape), tuple(lead)))


class _Call:
    """Device and stream of one call; new tensors are allocated for them."""

    __slots__ = ("dev", "handle", "stream")

    def __init__(self, first, inputs, others, stream):
        """`others`: integers and outputs, of which only the device matters."""
        try:
            dev = self.dev = first.get_device()
            grad = first.requires_grad
            for t in inputs:
                if t is not None:
                    if t.get_device() != dev:
                        raise TypeError(_DEVICES)
                    if t.requires_grad:
                        grad = True
            for t in others:
                if t is not None and t.get_device() != dev:
                    raise TypeError(_DEVICES)
        except AttributeError:
            raise TypeError("the operators take torch tensors") from None
        if dev < 0 or not first.is_cuda:
            raise TypeError("the operators take CUDA tensors")
        if grad and _is_grad_enabled():
            raise RuntimeError("the operators are not recorded by autograd: with a tensor that requires a gradient, "
                               "call them under torch.no_grad() or from a torch.autograd.Function")
        self.stream = None
        if stream is None:
            self.handle = _raw_stream(dev)
        else:
            self.handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
            if self.handle != _raw_stream(dev):
                if not isinstance(stream, torch.cuda.Stream):
                    stream = torch.cuda.ExternalStream(self.handle, device=dev)
                self.stream = stream
                # Not for streams of others' making, which may be gone when a tensor is freed.
                if not isinstance(stream, torch.cuda.ExternalStream):
                    for t in (first, *inputs, *others):
                        if t is not None:
                            t.record_stream(stream)

    def empty(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.dev))
        # From the pool of the stream that uses it: memory of another stream's
        # pool might still be in use there.
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.dev))

    def workspace(self, size):
        """(tensor, address) of scratch memory for one call.  Calls of one
        thread on one stream follow each other and share it; it grows to the
        largest asked for and goes with its thread.  A captured call gets memory
        of its own graph's."""
        if self.stream is not None or _is_capturing():
            t = self.empty((size,), torch.uint8)
            return t, t.data_ptr()
        key = (self.dev, self.handle, threading.get_ident())
        got = _workspaces.get(key)
        if got is None or got[2] < size:
            t = self.empty((size,), torch.uint8)
            _drop_with_thread(key[2])
            got = _workspaces[key] = (t, t.data_ptr(), size)
        return got[0], got[1]

    def run(self, name, written, *args):
        """The library's call; `written`: the tensors that it writes."""
        fn = (_fns or _load())[name]
        if self.dev == _current_device():
            code = fn(*args)
        else:
            with torch.cuda.device(self.dev):
                code = fn(*args)
        if code:
            _lopt._check(name, code)
        _increment_version(written)


_workspaces = {}         # (device, stream, thread): (tensor, address, size)
_local = threading.local()


class _End:
    """Goes with the thread it is a local of."""


def _drop(thread):
    for key in [k for k in list(_workspaces) if k[2] == thread]:
        _workspaces.pop(key, None)


def _drop_with_thread(thread):
    """Scratch memory of the calling thread goes when it ends."""
    if not hasattr(_local, "end"):
        _local.end = _End()
        weakref.finalize(_local.end, _drop, thread).atexit = False


def release_workspaces() -> None:
    """Give the operators' scratch memory, of all threads, back to torch's allocator."""
    _workspaces.clear()


@functools.lru_cache(maxsize=1024)
def _size_of(name, *sizes):
    """What a workspace function of the library says for these sizes."""
    need = ctypes.c_int64()
    code = _load()[name](*sizes, need)
    if code:
        _lopt._check(name, code)
    return need.value


_status = {}


def _status_ptr(dev):
    """Address of the library's status word on a device: the same for every
    thread, and there before the first call, be it a captured one."""
    ptr = _status.get(dev)
    if ptr is None:
        word = ctypes.c_void_p()
        with torch.cuda.device(dev):
            code = _load()["lopt_status_word"](word)
        if code:
            _lopt._check("lopt_status_word", code)
        ptr = _status[dev] = word.value
    return ptr


def check_indices(device: Optional[int] = None) -> None:
    """Wait for the device and raise LoptError (LOPT_E_INDEX) if an index of
    any call since the last check, replayed graphs among them, was at or above
    its limit (or LOPT_E_TIMEOUT if a kernel's bounded wait ran out)."""
    dev = torch.cuda.current_device() if device is None else torch.device("cuda", device).index
    if dev not in _status:
        return
    flags = ctypes.c_int32()
    with torch.cuda.device(dev):
        code = _load()["lopt_status_take"](flags)
    if code:
        _lopt._check("lopt_status_take", code)
    if flags.value:
        _lopt._check("check_indices", _E_TIMEOUT if flags.value & 2 else E_INDEX)


# ---- embedding ------------------------------------------------------------------


def embedding_forward(table, index, scale: float = 1.0, *, out=None, out_dtype=None, stream=None):
    """``out[i] = scale * table[index[i]]``, zeros where index[i] is negative.

    table: [rows, cols], float32, float16 or bfloat16; index: int32 or int64
    of any shape, contiguous; out: [*index.shape, cols] (default: new, of
    ``out_dtype`` or the table's type)."""
    c = _Call(table, (), (index, out), stream)
    if table.dim() != 2:
        raise ValueError("table must have two dimensions")
    rows, cols, ts = _matrix(table, "table")
    kind, n = _index(index, "index"), index.numel()
    if out is None:
        out = c.empty((*index.shape, cols), out_dtype or table.dtype)
    n_out, cols_out, os = _matrix(out, "out")
    if n_out != n or cols_out != cols:
        raise ValueError("out must be %s" % ((*index.shape, cols),))
    if out_dtype is not None and out.dtype is not out_dtype:
        raise TypeError("out is %s, out_dtype %s" % (out.dtype, out_dtype))
    if index.dim() > 1:
        _same_lead(index.shape, out=(out, 1))
    c.run("lopt_embed_forward", (out,), table.data_ptr(), _type(table, "table"), rows, cols, ts, index.data_ptr(),
          kind, n, scale, out.data_ptr(), _type(out, "out"), os, _status_ptr(c.dev), c.handle)
    return out


def embedding_backward(grad_out, index, rows: int, scale: float = 1.0, *, out=None, accumulate: bool = False,
                       stream=None):
    """The gradient of the table: float32 [rows, cols], row v the sum of
    ``scale * grad_out[i]`` over the i with index[i] == v, in that order.
    ``out``: the parameter's gradient buffer; ``accumulate`` adds to it (a
    table tied to the output projection) instead of writing every row."""
    c = _Call(grad_out, (), (index, out), stream)
    n, cols, gs = _matrix(grad_out, "grad_out")
    kind = _index(index, "index")
    if index.numel() != n:
        raise ValueError("grad_out has %d rows for %d indices" % (n, index.numel()))
    if index.dim() > 1:
        _same_lead(index.shape, grad_out=(grad_out, 1))
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = c.empty((rows, cols), torch.float32)
    elif out.shape != (rows, cols) and out.dim() != 1:
        raise ValueError("out must be %s" % ((rows, cols),))
    ptr = _vector(out, rows * cols, "out")
    need = _size_of("lopt_embed_workspace", n, rows, cols)
    ws, ws_ptr = c.workspace(need)
    c.run("lopt_embed_backward", (out,), grad_out.data_ptr(), _type(grad_out, "grad_out"), gs, index.data_ptr(),
          kind, n, rows, cols, scale, 1 if accumulate else 0, ptr, ws_ptr, need, _status_ptr(c.dev), c.handle)
    return out


# ---- layer norm -------------------------------------------------------------------


def _weight_type(weight, bias, x, cols):
    dtype = weight.dtype
    if dtype is not torch.float32 and dtype is not x.dtype:
        raise TypeError("weight must be float32 or of the type of x")
    w = _vector(weight, cols, "weight", dtype)
    return w, 0 if bias is None else _vector(bias, cols, "bias", dtype), _TYPES[dtype]


def _like(c, t, x, shape, what):
    """``t``, or a new tensor like x, with its address and row stride."""
    if t is None:
        t = c.empty(x.shape, x.dtype)
    rows, cols, stride = _matrix(t, what)
    if (rows, cols) != shape or t.dtype is not x.dtype:
        raise ValueError("%s must be %s of %s" % (what, tuple(x.shape), x.dtype))
    return t, t.data_ptr(), stride


def layernorm_forward(x, weight, bias=None, eps: float = 1e-5, *, residual=None, out=None, summed=None, mean=None,
                      rstd=None, stream=None):
    """Layer norm over the last dimension of x, or of x + residual.

    Returns (y, mean, rstd), or (y, summed, mean, rstd) with a residual:
    summed is x + residual, what the residual stream goes on with; mean and
    rstd (float32, one per row) are what the backward pass wants.  weight and
    bias: float32 or the type of x."""
    c = _Call(x, (weight, bias, residual), (out, summed, mean, rstd), stream)
    rows, cols, xs = _matrix(x, "x")
    if x.dim() > 2:
        _same_lead(x.shape[:-1], residual=(residual, 1), out=(out, 1), summed=(summed, 1), mean=(mean, 0),
                   rstd=(rstd, 0))
    kind = _type(x, "x")
    w, b, wt = _weight_type(weight, bias, x, cols)
    out, y, ys = _like(c, out, x, (rows, cols), "out")
    r = rs = s = ss = 0
    if residual is not None:
        residual, r, rs = _like(c, residual, x, (rows, cols), "residual")
        summed, s, ss = _like(c, summed, x, (rows, cols), "summed")
    elif summed is not None:
        raise ValueError("summed needs a residual")
    if mean is None:
        mean = c.empty(x.shape[:-1], torch.float32)
    if rstd is None:
        rstd = c.empty(x.shape[:-1], torch.float32)
    written = (out, mean, rstd) if residual is None else (out, summed, mean, rstd)
    c.run("lopt_layernorm_forward", written, x.data_ptr(), kind, rows, cols, xs, r, rs, w, b, wt, eps, y, ys, s, ss,
          _vector(mean, rows, "mean"), _vector(rstd, rows, "rstd"), c.handle)
    return written


def layernorm_backward(grad_out, x, mean, rstd, weight, *, grad_residual=None, need_bias: bool = True, grad_x=None,
                       grad_weight=None, grad_bias=None, accumulate: bool = False, stream=None):
    """The backward pass: (grad_x, grad_weight, grad_bias or None).

    x: the forward pass's x (or its ``summed``); grad_residual: the gradient
    that reaches x past the norm, added to grad_x; grad_weight and grad_bias:
    float32 [cols], the parameters' gradient buffers (``accumulate`` adds to
    them)."""
    c = _Call(grad_out, (x, weight, grad_residual), (mean, rstd, grad_x, grad_weight, grad_bias), stream)
    rows, cols, ds = _matrix(grad_out, "grad_out")
    if grad_out.dim() > 2:
        _same_lead(grad_out.shape[:-1], x=(x, 1), mean=(mean, 0), rstd=(rstd, 0), grad_residual=(grad_residual, 1),
                   grad_x=(grad_x, 1))
    kind = _type(grad_out, "grad_out")
    x, xp, xs = _like(c, x, grad_out, (rows, cols), "x")
    w, _, wt = _weight_type(weight, None, grad_out, cols)
    r = rs = 0
    if grad_residual is not None:
        grad_residual, r, rs = _like(c, grad_residual, grad_out, (rows, cols), "grad_residual")
    if accumulate and (grad_weight is None or (need_bias and grad_bias is None)):
        raise ValueError("accumulate needs grad_weight and grad_bias")
    grad_x, gx, gs = _like(c, grad_x, grad_out, (rows, cols), "grad_x")
    if grad_weight is None:
        grad_weight = c.empty((cols,), torch.float32)
    if not need_bias:
        grad_bias = None
    elif grad_bias is None:
        grad_bias = c.empty((cols,), torch.float32)
    need = _size_of("lopt_layernorm_workspace", rows, cols)
    ws, ws_ptr = c.workspace(need)
    written = (grad_x, grad_weight) if grad_bias is None else (grad_x, grad_weight, grad_bias)
    c.run("lopt_layernorm_backward", written, grad_out.data_ptr(), kind, rows, cols, ds, xp, xs,
          _vector(mean, rows, "mean"), _vector(rstd, rows, "rstd"), w, wt, r, rs, gx, gs,
          _vector(grad_weight, cols, "grad_weight"), 0 if grad_bias is None else _vector(grad_bias, cols, "grad_bias"),
          1 if accumulate else 0, ws_ptr, need, c.handle)
    return grad_x, grad_weight, grad_bias


# ---- distillation -----------------------------------------------------------------


def _distill(logits, top_logits, top_index, temperature, row_weight, loss, grad, need_grad, stream):
    c = _Call(logits, (top_logits, row_weight), (top_index, loss, grad), stream)
    rows, cols, zs = _matrix(logits, "logits")
    if logits.dim() > 2:
        _same_lead(logits.shape[:-1], top_logits=(top_logits, 1), top_index=(top_index, 1), row_weight=(row_weight, 0),
                   loss=(loss, 0), grad=(grad, 1))
    kind = _type(logits, "logits")
    t_rows, top, ts = _matrix(top_logits, "top_logits")
    i_rows, i_top, i_s = _matrix(top_index, "top_index")
    if t_rows != rows or (i_rows, i_top) != (rows, top):
        raise ValueError("top_logits and top_index must be [%d, top]" % rows)
    if top_logits.dtype is not logits.dtype and top_logits.dtype is not torch.float32:
        raise TypeError("top_logits must be float32 or of the type of the logits")
    ik = _INDEX.get(top_index.dtype)
    if ik is None:
        raise TypeError("top_index must be int32 or int64, not %s" % top_index.dtype)
    w = 0 if row_weight is None else _vector(row_weight, rows, "row_weight")
    if loss is None:
        loss = c.empty(logits.shape[:-1], torch.float32)
    g = gs = 0
    if need_grad:
        grad, g, gs = _like(c, grad, logits, (rows, cols), "grad")
    c.run("lopt_distill", (loss, grad) if need_grad else (loss,), logits.data_ptr(), kind, rows, cols, zs,
          top_logits.data_ptr(), _TYPES[top_logits.dtype], ts, top_index.data_ptr(), ik, i_s, top, temperature, w,
          _vector(loss, rows, "loss"), g, gs, _status_ptr(c.dev), c.handle)
    return loss, grad


def distill_forward(logits, top_logits, top_index, temperature: float = 1.0, *, row_weight=None, loss=None,
                    stream=None):
    """The loss of each row (float32): row_weight * T^2 * KL(p || q), p the
    teacher's softmax over the listed classes, q the softmax of the logits,
    both at temperature T (1e-30 to 1e3).

    logits: [..., classes]; top_logits, top_index: [..., top], top <= 1024;
    slots with a negative index or a logit of -inf do not count.  A row of
    weight 0, or without slots that count, has loss 0 whatever its logits
    hold.  With one slot per row it is the cross entropy with that class."""
    return _distill(logits, top_logits, top_index, temperature, row_weight, loss, None, False, stream)[0]


def distill_forward_backward(logits, top_logits, top_index, temperature: float = 1.0, *, row_weight=None, loss=None,
                             grad=None, stream=None):
    """(loss, grad): the loss of each row and the gradient of their sum with
    respect to the logits, in the logits' type and from one read of them.
    ``grad`` may be the logits themselves, which it then replaces."""
    return _distill(logits, top_logits, top_index, temperature, row_weight, loss, grad, True, stream)
