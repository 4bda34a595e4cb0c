"""Cases, plain forms and 64-bit results of the training operators.

Three operators stand between a model's matrix products and the learned
optimizer's step, which reads one contiguous float32 gradient per parameter:

  embedding     the first layer's lookup and the gradient of its table,
  layer norm    forward (with the residual sum before it) and backward
                (with the gradients of weight and bias),
  distillation  the loss against a teacher's top logits, with its gradient.

``own`` selects who computes a pass: False the plain form below (elementary
torch operations in float32, rounded once at the end), True the kernels of
learned_optimizer_step_gb300.  A training loop keeps its gradients, and here
also its activations, in buffers of its own: the state holds them and the
calls write into them.
"""

import math

import numpy as np
import torch

own = False

_DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16,
           "int32": torch.int32, "int64": torch.int64}
_SIZE = {"float32": 4, "float16": 2, "bfloat16": 2, "int32": 4, "int64": 8}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------


def listed():
    return [
        # Token by token: one new token for each of 16 sequences, looked up in
        # the float32 master table of the GPT-2-small list.
        {"name": "embed_fwd_16_tokens", "op": "embed_fwd", "tokens": 16, "rows": 50257, "cols": 768,
         "table": "float32", "dtype": "bfloat16", "index": "int64", "scale": 1.0, "padding": 0.0},
        # The first layer of a training step of the 1.3B decoder: 16 sequences
        # of 1024 tokens, activations scaled by the square root of the width.
        {"name": "embed_fwd_batch_2048", "op": "embed_fwd", "tokens": 16384, "rows": 50304, "cols": 2048,
         "table": "float32", "dtype": "bfloat16", "index": "int64", "scale": math.sqrt(2048.0), "padding": 0.0},
        # The table's gradient from a small ragged batch: sequences of
        # different lengths, padded; the padding carries no gradient.
        {"name": "embed_bwd_ragged", "op": "embed_bwd", "tokens": 4099, "rows": 50257, "cols": 768,
         "table": "float32", "dtype": "float16", "index": "int32", "scale": 1.0, "padding": 0.25},
        # The table's gradient of a large step of the 1.3B decoder.
        {"name": "embed_bwd_batch_2048", "op": "embed_bwd", "tokens": 65536, "rows": 50304, "cols": 2048,
         "table": "float32", "dtype": "bfloat16", "index": "int64", "scale": math.sqrt(2048.0), "padding": 0.0},
        # Token by token: the norm before the head for 16 sequences.
        {"name": "norm_fwd_16_rows", "op": "norm_fwd", "rows": 16, "cols": 768, "dtype": "float32",
         "weight": "float32", "bias": True, "residual": False},
        # A block's norm with the residual sum before it; the batch is packed
        # from sequences of different lengths, so the row count is odd.
        {"name": "norm_fwd_residual_768", "op": "norm_fwd", "rows": 16421, "cols": 768, "dtype": "bfloat16",
         "weight": "float32", "bias": True, "residual": True},
        # The same width's backward pass in float16, a small batch.
        {"name": "norm_bwd_768", "op": "norm_bwd", "rows": 2047, "cols": 768, "dtype": "float16",
         "weight": "float32", "bias": True, "residual": False},
        # Backward in the 1.3B decoder, joined with the residual's gradient.
        {"name": "norm_bwd_residual_2048", "op": "norm_bwd", "rows": 32768, "cols": 2048, "dtype": "bfloat16",
         "weight": "float32", "bias": True, "residual": True},
        # A micro-batch of answers: seven tokens over the whole vocabulary.
        {"name": "distill_7_tokens", "op": "distill", "rows": 7, "cols": 50257, "top": 64, "dtype": "bfloat16",
         "teacher": "float32", "index": "int64", "temperature": 2.0, "masked": 0.0, "nucleus": False, "grad": True},
        # An image classifier's head (1000 classes) learning a teacher's top
        # classes, softened.
        {"name": "distill_1000_classes", "op": "distill", "rows": 4096, "cols": 1000, "top": 20, "dtype": "float32",
         "teacher": "float32", "index": "int64", "temperature": 4.0, "masked": 0.0, "nucleus": False, "grad": True},
        # A training step over the GPT-2-small vocabulary: loss and gradient
        # of 8192 tokens; prompts do not count, and the teacher's list ends
        # where its probability is spent.
        {"name": "distill_batch_50257", "op": "distill", "rows": 8192, "cols": 50257, "top": 64, "dtype": "bfloat16",
         "teacher": "bfloat16", "index": "int32", "temperature": 1.0, "masked": 0.125, "nucleus": True, "grad": True},
        # Evaluation: the loss alone.
        {"name": "distill_loss_only", "op": "distill", "rows": 2048, "cols": 50304, "top": 128, "dtype": "float16",
         "teacher": "float16", "index": "int32", "temperature": 1.0, "masked": 0.125, "nucleus": True, "grad": False},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "distill"])
    half = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    if op.startswith("embed"):
        cols = _spread(rng, 64, 2048)
        cols = cols if rng.random() < 0.3 else cols // 8 * 8
        return {"op": op, "tokens": _spread(rng, 1, 65536), "rows": _spread(rng, 300, 65536), "cols": cols,
                "table": "float32", "dtype": half, "index": rng.choice(["int32", "int64"]),
                "scale": rng.choice([1.0, math.sqrt(cols)]), "padding": rng.choice([0.0, 0.25])}
    if op.startswith("norm"):
        cols = _spread(rng, 64, 8192)
        cols = cols if rng.random() < 0.3 else cols // 8 * 8
        rows = _spread(rng, 1, min(32768, 32768 * 2048 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": half, "weight": rng.choice(["float32", half]),
                "bias": rng.random() < 0.8, "residual": rng.random() < 0.5}
    cols = _spread(rng, 200, 131072)
    rows = _spread(rng, 1, min(8192, 8192 * 50257 // cols))
    return {"op": op, "rows": rows, "cols": cols, "top": _spread(rng, 1, 128), "dtype": half,
            "teacher": rng.choice(["float32", half]), "index": rng.choice(["int32", "int64"]),
            "temperature": rng.choice([1.0, 2.0, 4.0]), "masked": rng.choice([0.0, 0.125]),
            "nucleus": rng.random() < 0.5, "grad": rng.random() < 0.75}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------


def _tokens(g, count, rows, dtype, padding):
    """Token ids as text has them: the chance of id v falls as 1/(v + 1)."""
    u = torch.rand(count, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(rows + 1.0)) - 1.0).long().clamp_(0, rows - 1)
    if padding:
        order = torch.rand(count, generator=g, device="cuda")
        ids[order < padding] = -1
    return ids.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = dict(case)
    op = case["op"]
    if op.startswith("embed"):
        n, rows, cols = case["tokens"], case["rows"], case["cols"]
        s["index"] = _tokens(g, n, rows, _DTYPES[case["index"]], case["padding"])
        if op == "embed_fwd":
            s["table"] = normal(rows, cols, std=0.02)
            s["out"] = empty(n, cols, dtype=dt)
        else:
            s["grad_out"] = normal(n, cols, std=1e-3, dtype=dt)
            s["out"] = empty(rows, cols)
    elif op.startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        wt = _DTYPES[case["weight"]]
        # Features of a residual stream: scales that differ from column to
        # column and a mean away from zero.
        scale = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
        x = torch.randn(rows, cols, generator=g, device="cuda") * scale + 0.1
        s["x"] = x.to(dt)
        s["weight"] = normal(cols, std=0.1, mean=1.0, dtype=wt)
        s["bias"] = normal(cols, std=0.1, dtype=wt) if case["bias"] else None
        s["mean"], s["rstd"] = empty(rows), empty(rows)
        s["out"] = empty(rows, cols, dtype=dt)
        if op == "norm_fwd":
            s["residual"] = normal(rows, cols, std=0.5, dtype=dt) if case["residual"] else None
            s["summed"] = empty(rows, cols, dtype=dt) if case["residual"] else None
        else:
            f = s["x"].float()
            s["mean"] = f.mean(1)
            s["rstd"] = torch.rsqrt(f.var(1, unbiased=False) + 1e-5)
            s["grad_out"] = normal(rows, cols, std=1e-2, dtype=dt)
            s["grad_residual"] = normal(rows, cols, std=1e-2, dtype=dt) if case["residual"] else None
            s["grad_weight"] = empty(cols)
            s["grad_bias"] = empty(cols) if case["bias"] else None
    else:
        rows, cols = case["rows"], case["cols"]
        top = min(case["top"], cols)
        s["logits"] = empty(rows, cols, dtype=dt)
        values, index = empty(rows, top), empty(rows, top, dtype=torch.int64)
        step = max(1, (1 << 26) // cols)
        for r in range(0, rows, step):
            base = torch.randn(min(step, rows - r), cols, generator=g, device="cuda") * 2.0
            s["logits"][r:r + step] = (base + 0.7 * torch.randn(base.shape, generator=g, device="cuda")).to(dt)
            values[r:r + step], index[r:r + step] = torch.topk(base * 1.5, top, dim=1)
        if case["nucleus"]:  # the teacher's list ends at 0.95 of its top probability
            p = torch.softmax(values, 1)
            index[p.cumsum(1) - p > 0.95] = -1
        s["top_logits"] = values.to(_DTYPES[case["teacher"]])
        s["top_index"] = index.to(_DTYPES[case["index"]])
        # The mean over the rows; in float16 their sum, as a loss scale of
        # `rows` makes it, so that the gradients stay within its range.
        s["row_weight"] = torch.full((rows,), 1.0 if dt == torch.float16 else 1.0 / rows, device="cuda")
        s["row_weight"][:int(case["masked"] * rows)] = 0.0
        s["loss"] = empty(rows)
        s["out"] = empty(rows, cols, dtype=dt) if case["grad"] else None
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import learned_optimizer_step_gb300 as L
    op = s["op"]
    if op == "embed_fwd":
        return L.embedding_forward(s["table"], s["index"], s["scale"], out=s["out"])
    if op == "embed_bwd":
        return L.embedding_backward(s["grad_out"], s["index"], s["rows"], s["scale"], out=s["out"])
    if op == "norm_fwd":
        return L.layernorm_forward(s["x"], s["weight"], s["bias"], 1e-5, residual=s["residual"], out=s["out"],
                                   summed=s["summed"], mean=s["mean"], rstd=s["rstd"])
    if op == "norm_bwd":
        return L.layernorm_backward(s["grad_out"], s["x"], s["mean"], s["rstd"], s["weight"],
                                    grad_residual=s["grad_residual"], need_bias=s["bias"] is not None,
                                    grad_x=s["out"], grad_weight=s["grad_weight"], grad_bias=s["grad_bias"])
    if not s["grad"]:
        return L.distill_forward(s["logits"], s["top_logits"], s["top_index"], s["temperature"],
                                 row_weight=s["row_weight"], loss=s["loss"])
    return L.distill_forward_backward(s["logits"], s["top_logits"], s["top_index"], s["temperature"],
                                      row_weight=s["row_weight"], loss=s["loss"], grad=s["out"])


def _plain(s):
    op = s["op"]
    dt = _DTYPES[s["dtype"]]
    if op == "embed_fwd":
        index = s["index"].long()
        rows = s["table"][index.clamp(min=0)].float() * s["scale"]
        return torch.where((index >= 0)[:, None], rows, 0.0).to(dt)
    if op == "embed_bwd":
        index = s["index"].long()
        grads = torch.where((index >= 0)[:, None], s["grad_out"].float() * s["scale"], 0.0)
        out = torch.zeros(s["rows"], s["cols"], device="cuda")
        return out.index_add_(0, index.clamp(min=0), grads)
    if op == "norm_fwd":
        x = s["x"].float()
        if s["residual"] is not None:
            x = x + s["residual"].float()
        mean = x.sum(1) / x.shape[1]
        d = x - mean[:, None]
        rstd = torch.rsqrt((d * d).sum(1) / x.shape[1] + 1e-5)
        y = d * rstd[:, None] * s["weight"].float()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        if s["residual"] is not None:
            return y.to(dt), x.to(dt), mean, rstd
        return y.to(dt), mean, rstd
    if op == "norm_bwd":
        dy = s["grad_out"].float()
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["weight"].float()
        n = dy.shape[1]
        a, b = g.sum(1) / n, (g * xhat).sum(1) / n
        dx = s["rstd"][:, None] * (g - a[:, None] - xhat * b[:, None])
        if s["grad_residual"] is not None:
            dx = dx + s["grad_residual"].float()
        return dx.to(dt), (dy * xhat).sum(0), dy.sum(0) if s["bias"] is not None else None
    T, w = s["temperature"], s["row_weight"]
    z = s["logits"].float() / T
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    index = s["top_index"].long()
    t = torch.where(index >= 0, s["top_logits"].float() / T, -math.inf)
    t = t - t.amax(1, keepdim=True)
    p = torch.exp(t)
    total = p.sum(1, keepdim=True)
    p = p / total
    index = index.clamp(min=0)
    terms = p * (t - torch.log(total) - torch.gather(z, 1, index) + lse[:, None])
    loss = T * T * w * torch.where(p > 0, terms, 0.0).sum(1)
    if not s["grad"]:
        return loss
    q = torch.exp(z - lse[:, None]).scatter_add_(1, index, -p)
    return loss, (q * (T * w)[:, None]).to(dt)


# --------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# --------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    f64 = torch.float64
    if op == "embed_fwd":
        index = s["index"].long()
        out = torch.zeros(s["tokens"], s["cols"], dtype=f64, device="cuda")
        real = index >= 0
        out[real] = torch.index_select(s["table"], 0, index[real]).to(f64).mul_(s["scale"])
        return out
    if op == "embed_bwd":
        index = s["index"].long()
        real = index >= 0
        out = torch.zeros(s["rows"], s["cols"], dtype=f64, device="cuda")
        out.index_put_((index[real],), s["grad_out"][real].to(f64), accumulate=True)
        return out.mul_(s["scale"])
    if op == "norm_fwd":
        x = s["x"].to(f64)
        if s["residual"] is not None:
            x = x + s["residual"].to(f64)
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + 1e-5).pow(-0.5)
        y = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1) * s["weight"].to(f64)
        y = y if s["bias"] is None else y + s["bias"].to(f64)
        return (y, mean, rstd) if s["residual"] is None else (y, x, mean, rstd)
    if op == "norm_bwd":
        # The derivative of sum(y * grad_out) with mean and variance written
        # out: dx = rstd * (I - 1/n - xhat xhat' / n) (weight * grad_out).
        dy, n = s["grad_out"].to(f64), s["cols"]
        rstd = s["rstd"].to(f64).unsqueeze(1)
        xhat = (s["x"].to(f64) - s["mean"].to(f64).unsqueeze(1)) * rstd
        v = dy * s["weight"].to(f64)
        dx = rstd * (v - v.mean(1, keepdim=True) - xhat * (v * xhat).mean(1, keepdim=True))
        if s["grad_residual"] is not None:
            dx = dx + s["grad_residual"].to(f64)
        return dx, torch.einsum("rc,rc->c", dy, xhat), dy.sum(0) if s["bias"] is not None else None
    T, rows, cols = s["temperature"], s["rows"], s["cols"]
    loss = torch.zeros(rows, dtype=f64, device="cuda")
    grad = torch.zeros(rows, cols, dtype=f64, device="cuda") if s["grad"] else None
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        part = slice(r, min(r + step, rows))
        logq = torch.log_softmax(s["logits"][part].to(f64) / T, 1)
        index = s["top_index"][part].long()
        t = s["top_logits"][part].to(f64) / T
        t[index < 0] = -math.inf
        logp = torch.log_softmax(t, 1)
        p = torch.zeros_like(logq).scatter_add_(1, index.clamp(min=0), logp.exp())
        at = logq.gather(1, index.clamp(min=0))
        w = s["row_weight"][part].to(f64)
        loss[part] = w * T * T * (logp.exp() * torch.where(index < 0, 0.0, logp - at)).sum(1)
        if grad is not None:
            grad[part] = (logq.exp() - p) * (w * T).unsqueeze(1)
    return loss if grad is None else (loss, grad)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------


def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op.startswith("embed"):
        n, rows, cols = case["tokens"], case["rows"], case["cols"]
        real = n * (1.0 - case["padding"])
        ids = n * _SIZE[case["index"]]
        if op == "embed_bwd":
            return {"bytes": ids + real * cols * e + rows * cols * 4, "flops": real * cols}
        v = np.arange(rows, dtype=np.float64)
        p = np.log((v + 2.0) / (v + 1.0)) / math.log(rows + 1.0)
        touched = float((1.0 - np.power(1.0 - p, real)).sum())  # different rows of the table, expected
        return {"bytes": ids + touched * cols * 4 + n * cols * e, "flops": real * cols}
    if op.startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        w = cols * _SIZE[case["weight"]]
        if op == "norm_fwd":
            arrays = 4 if case["residual"] else 2
            return {"bytes": rows * cols * e * arrays + w * (1 + case["bias"]) + 8 * rows, "flops": 8.0 * rows * cols}
        arrays = 4 if case["residual"] else 3
        return {"bytes": rows * cols * e * arrays + w + 4 * cols * (1 + case["bias"]) + 8 * rows,
                "flops": 14.0 * rows * cols}
    rows, cols, top = case["rows"], case["cols"], min(case["top"], case["cols"])
    counted = rows - int(case["masked"] * rows)
    lists = counted * top * (_SIZE[case["teacher"]] + _SIZE[case["index"]])
    grads = rows * cols * e if case["grad"] else 0
    return {"bytes": counted * cols * e + grads + lists + 8 * rows,
            "flops": (5.0 if case["grad"] else 3.0) * counted * cols}
