"""Cases, plain forms and 64-bit results of the language model's training operators.

Three operators around a language model's blocks, its loss and its weights:

  block norm      what stands between two blocks: the norm of a block's output,
                  its gate and residual scale, the sum with the residual
                  stream, and the norm before the next block; and its backward
                  pass,
  cross entropy   of the next token over a large vocabulary, from the hidden
                  states and the output table without keeping the logits; and
                  its backward pass,
  AdamW           one step over a whole list of tensors, moments in 32 bits or
                  in 8, with the gradients clipped by their global norm.

``own`` selects who computes a pass: False the plain form below (elementary
torch operations in float32, rounded once at the end), True the kernels of
learned_optimizer_step_gb300.  A training loop keeps its gradients, activations
and moments in buffers of its own: the state holds them and the calls write
into them.
"""

import math
import random

import torch

own = False

_DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16,
           "int32": torch.int32, "int64": torch.int64}
_SIZE = {"float32": 4, "float16": 2, "bfloat16": 2, "int32": 4, "int64": 8}

_EPS_NORM = 1e-6
_BETA1, _BETA2, _EPS, _DECAY, _LR = 0.9, 0.999, 1e-8, 0.1, 3e-4
_BLOCK = 256          # elements that share a scale of 8-bit moments
_TOP_M, _TOP_V = 127, 255


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------


def listed():
    return [
        # Scoring: the log probabilities of seven tokens under the
        # GPT-2-small vocabulary and width.
        {"name": "loss_7_tokens", "op": "loss", "rows": 7, "classes": 50257, "cols": 768, "dtype": "bfloat16",
         "index": "int64", "padding": 0.0},
        # Evaluation of the 1.3B decoder: 4 sequences of 2048 tokens, a few
        # of them padding.
        {"name": "loss_batch_2048", "op": "loss", "rows": 8192, "classes": 50304, "cols": 2048, "dtype": "float16",
         "index": "int32", "padding": 0.0625},
        # A small ragged batch of the example's model: gradients in the type
        # of the activations.
        {"name": "loss_bwd_ragged_256", "op": "loss_bwd", "rows": 203, "classes": 5003, "cols": 256,
         "dtype": "bfloat16", "index": "int64", "padding": 0.125, "grad": "bfloat16"},
        # The GPT-2-small head in float16; its table's gradient goes to the
        # optimizer in float32.
        {"name": "loss_bwd_768", "op": "loss_bwd", "rows": 4099, "classes": 50257, "cols": 768, "dtype": "float16",
         "index": "int32", "padding": 0.0, "grad": "float32"},
        # A training step of the 1.3B decoder's head.
        {"name": "loss_bwd_batch_2048", "op": "loss_bwd", "rows": 8192, "classes": 50304, "cols": 2048,
         "dtype": "bfloat16", "index": "int64", "padding": 0.0, "grad": "float32"},
        # The example's small model: some ten tensors, where latency counts.
        {"name": "adamw_small", "op": "adamw", "list": "decoder", "classes": 5003, "cols": 256, "layers": 1,
         "moments": "float32", "grad": "float32", "copy": "none", "clip": True, "align": 256},
        # The whole 1.3B decoder, 291 tensors, with the bfloat16 copy of the
        # weights that the next step's products read.
        {"name": "adamw_1p3b", "op": "adamw", "list": "decoder", "classes": 50304, "cols": 2048, "layers": 24,
         "moments": "float32", "grad": "float32", "copy": "bfloat16", "clip": True, "align": 256},
        # Four of its layers with 8-bit moments and bfloat16 gradients.
        {"name": "adamw_8bit", "op": "adamw", "list": "decoder", "classes": 50304, "cols": 2048, "layers": 4,
         "moments": "8bit", "grad": "bfloat16", "copy": "bfloat16", "clip": False, "align": 256},
        # Token by token: one new token for each of 16 sequences.
        {"name": "norm_fwd_16_rows", "op": "norm_fwd", "rows": 16, "cols": 2048, "dtype": "bfloat16",
         "weight": "float32", "gate": True},
        # A batch packed from sequences of different lengths.
        {"name": "norm_fwd_768", "op": "norm_fwd", "rows": 16421, "cols": 768, "dtype": "bfloat16",
         "weight": "float32", "gate": True},
        # A small batch backward, in float16.
        {"name": "norm_bwd_768", "op": "norm_bwd", "rows": 2047, "cols": 768, "dtype": "float16",
         "weight": "float32", "gate": True},
        # Backward in the 1.3B decoder, without gates.
        {"name": "norm_bwd_2048", "op": "norm_bwd", "rows": 32768, "cols": 2048, "dtype": "bfloat16",
         "weight": "float32", "gate": False},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["loss", "loss_bwd", "loss_bwd", "adamw", "adamw", "norm_fwd", "norm_bwd"])
    half = rng.choice(["bfloat16", "bfloat16", "float16"])
    if op.startswith("loss"):
        cols = _spread(rng, 64, 2048)
        cols = cols if rng.random() < 0.2 else max(8, cols // 8 * 8)
        classes = _spread(rng, 300, 131072)
        most = 8192 * 50304 * 2048 // (classes * cols)
        case = {"op": op, "rows": _spread(rng, 1, max(2, min(8192, most))), "classes": classes, "cols": cols,
                "dtype": half, "index": rng.choice(["int32", "int64"]), "padding": rng.choice([0.0, 0.125])}
        if op == "loss_bwd":
            case["grad"] = rng.choice(["float32", half])
        return case
    if op == "adamw":
        moments = rng.choice(["float32", "8bit"])
        return {"op": op, "list": "ragged", "tensors": _spread(rng, 1, 300), "largest": _spread(rng, 1000, 4000000),
                "shapes": rng.randrange(1 << 30), "moments": moments,
                "grad": rng.choice(["float32", "float32", "bfloat16", "float16"]),
                "copy": rng.choice(["none", "bfloat16", "float16"]), "clip": rng.random() < 0.5,
                "align": 256 if moments == "8bit" else rng.choice([1, 256])}
    cols = _spread(rng, 64, 8192)
    cols = cols if rng.random() < 0.3 else cols // 8 * 8
    half = rng.choice([half, half, "float32"])
    rows = _spread(rng, 1, min(32768, 32768 * 2048 // cols))
    return {"op": op, "rows": rows, "cols": cols, "dtype": half, "weight": rng.choice(["float32", half]),
            "gate": rng.random() < 0.5}


def _layout(case):
    """The tensors of a list in one flat buffer: (offset, elements, whether
    weight decay applies) each, those with decay first, and how many elements
    those take and all do."""
    if case["list"] == "decoder":
        d, matrices, vectors = case["cols"], [case["classes"] * case["cols"]], []
        for _ in range(case["layers"]):
            matrices += [3 * d * d, d * d, 4 * d * d, 4 * d * d]
            vectors += [3 * d, d, 4 * d, d, d, d, d, d]
        vectors += [d, d]
    else:
        r = random.Random(case["shapes"])
        sizes = [_spread(r, 1, case["largest"]) for _ in range(case["tensors"])]
        matrices, vectors = sizes[::2], sizes[1::2]
    at, out = 0, []
    decayed = 0
    for n, decay in [(n, True) for n in matrices] + [(n, False) for n in vectors]:
        out.append((at, n, decay))
        at += -(-n // case["align"]) * case["align"]
        decayed = at if decay else decayed
    return out, decayed, at


def work(case):
    op = case["op"]
    if op.startswith("loss"):
        n, v, d, es = case["rows"], case["classes"], case["cols"], _SIZE[case["dtype"]]
        inputs = (n + v) * d * es + n * _SIZE[case["index"]]
        if op == "loss":
            return {"bytes": inputs + 8 * n, "flops": 2 * n * v * d}
        return {"bytes": inputs + 8 * n + n * d * es + v * d * _SIZE[case["grad"]], "flops": 6 * n * v * d}
    if op == "adamw":
        n = sum(t[1] for t in _layout(case)[0])
        each = 8 + _SIZE[case["grad"]] + (_SIZE[case["copy"]] if case["copy"] != "none" else 0)
        # 8-bit moments: also written out as the values they stand for.
        each += 16 if case["moments"] == "float32" else 4 + 16 / _BLOCK + 8
        return {"bytes": int(n * each), "flops": 12 * n}
    n, es, cols = case["rows"] * case["cols"], _SIZE[case["dtype"]], case["cols"]
    if op == "norm_fwd":
        return {"bytes": n * es * (4 + case["gate"]) + 8 * case["rows"] + 2 * cols * _SIZE[case["weight"]],
                "flops": 10 * n}
    return {"bytes": n * es * (6 + 2 * case["gate"]) + 8 * case["rows"] + 2 * cols * (_SIZE[case["weight"]] + 4),
            "flops": 20 * n}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------


def _tokens(g, count, classes, dtype, padding):
    """Token ids as text has them: the chance of id v falls as 1/(v + 1)."""
    u = torch.rand(count, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(classes + 1.0)) - 1.0).long().clamp_(0, classes - 1)
    if padding:
        order = torch.rand(count, generator=g, device="cuda")
        ids[order < padding] = -1
    return ids.to(dtype)


def _tensor_key(seed, index):
    return _scramble(seed ^ ((index + 1) * 0x9E3779B9 & 0xFFFFFFFF))


def _scramble(h):
    """The final mixing of MurmurHash3's 32-bit variant; ints or int64 tensors."""
    h = h ^ (h >> 16)
    h = h * 0x85EBCA6B & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = h * 0xC2B2AE35 & 0xFFFFFFFF
    return h ^ (h >> 16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = dict(case)
    op = case["op"]
    if op == "adamw":
        s["layout"], s["decayed"], size = _layout(case)
        used = torch.zeros(size, device="cuda")       # 1 where a tensor has an element
        for at, n, _ in s["layout"]:
            used[at:at + n] = 1.0
        s["param"] = normal(size, std=0.02).mul_(used)
        s["gradient"] = normal(size, std=1e-3).mul_(used).to(_DTYPES[case["grad"]])
        s["copied"] = None if case["copy"] == "none" else s["param"].to(_DTYPES[case["copy"]])
        s["step"], s["seed"] = 1000, int(seed) & 0xFFFFFFFF
        # Often above the clip's limit, as early in a training run.
        s["max_norm"] = 5e-4 * math.sqrt(sum(t[1] for t in s["layout"])) if case["clip"] else None
        if case["moments"] == "float32":
            s["m"] = normal(size, std=3e-4).mul_(used)
            s["v"] = normal(size, std=1e-3).square_().mul_(used)
        else:
            blocks = size // _BLOCK
            s["m_codes"] = normal(size, std=40.0).clamp_(-_TOP_M, _TOP_M).mul_(used).to(torch.int8)
            s["v_codes"] = (normal(size, std=40.0).abs_().clamp_(0, 200.0) + 30.0).mul_(used).to(torch.uint8)
            s["m_scale"] = torch.exp(normal(blocks, std=0.5)) * (1e-3 / _TOP_M ** 2)
            s["v_scale"] = torch.exp(normal(blocks, std=0.5)) * (3e-3 / _TOP_V ** 2)
            s["m"], s["v"] = torch.zeros(size, device="cuda"), torch.zeros(size, device="cuda")
            # For the plain form: every element's random number comes from
            # its tensor's key and its place in the tensor.
            keys = torch.zeros(blocks, dtype=torch.int64)
            first = torch.zeros(blocks, dtype=torch.int64)
            for k, (at, n, _) in enumerate(s["layout"]):
                here = slice(at // _BLOCK, (at + n + _BLOCK - 1) // _BLOCK)
                keys[here] = _tensor_key(s["seed"], k)
                first[here] = torch.arange(here.stop - here.start) * _BLOCK
            s["keys"], s["first"] = keys.cuda(), first.cuda()
        return s
    dt = _DTYPES[case["dtype"]]
    rows, cols = case["rows"], case["cols"]
    if op.startswith("loss"):
        classes = case["classes"]
        s["table"] = normal(classes, cols, std=1.0 / math.sqrt(cols), dtype=dt)
        s["target"] = _tokens(g, rows, classes, _DTYPES[case["index"]], case["padding"])
        # Hidden states that know something of the next token.
        known = torch.rand(rows, 1, generator=g, device="cuda") * 16.0
        x = torch.randn(rows, cols, generator=g, device="cuda")
        s["x"] = (x + known * s["table"][s["target"].long().clamp(min=0)].float()).to(dt)
        # The mean over the rows; in float16 their sum, as a loss scale of
        # `rows` makes it, so that the gradients stay within its range.
        s["row_weight"] = torch.full((rows,), 1.0 if dt == torch.float16 else 1.0 / rows, device="cuda")
        s["loss"], s["lse"] = empty(rows), empty(rows)
        if op == "loss_bwd":
            _plain_loss(s)
            s["lse"] = s["lse"].clone()
            s["grad_x"] = empty(rows, cols, dtype=dt)
            s["grad_table"] = empty(classes, cols, dtype=_DTYPES[case["grad"]])
        return s
    wt = _DTYPES[case["weight"]]
    # A block's output and the residual stream: scales that differ from column
    # to column.
    h = torch.randn(rows, cols, generator=g, device="cuda")
    s["h"] = (h * torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))).to(dt)
    s["residual"] = normal(rows, cols, std=2.0, dtype=dt)
    s["gate"] = normal(rows, cols, std=1.5, dtype=dt) if case["gate"] else None
    s["w_post"] = normal(cols, std=0.1, mean=1.0, dtype=wt)
    s["w_pre"] = normal(cols, std=0.1, mean=1.0, dtype=wt)
    s["scale"] = 0.7
    s["rstd_post"], s["rstd_pre"] = empty(rows), empty(rows)
    s["out"], s["summed"] = empty(rows, cols, dtype=dt), empty(rows, cols, dtype=dt)
    if op == "norm_bwd":
        _, s["summed"], s["rstd_post"], s["rstd_pre"] = _plain_norm(s)
        del s["residual"]
        s["grad_out"] = normal(rows, cols, std=1e-2, dtype=dt)
        s["grad_summed"] = normal(rows, cols, std=1e-2, dtype=dt)
        s["grad_h"], s["grad_residual"] = empty(rows, cols, dtype=dt), empty(rows, cols, dtype=dt)
        s["grad_gate"] = empty(rows, cols, dtype=dt) if case["gate"] else None
        s["grad_w_post"], s["grad_w_pre"] = empty(cols), empty(cols)
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import learned_optimizer_step_gb300 as L
    op = s["op"]
    if op == "loss":
        return L.linear_cross_entropy_forward(s["x"], s["table"], s["target"], row_weight=s["row_weight"],
                                              loss=s["loss"], lse=s["lse"])
    if op == "loss_bwd":
        return L.linear_cross_entropy_backward(s["x"], s["table"], s["target"], s["lse"], row_weight=s["row_weight"],
                                               grad_x=s["grad_x"], grad_weight=s["grad_table"])
    if op == "norm_fwd":
        return L.block_norm_forward(s["h"], s["residual"], s["w_post"], s["w_pre"], gate=s["gate"], scale=s["scale"],
                                    eps=_EPS_NORM, out=s["out"], summed=s["summed"], rstd_post=s["rstd_post"],
                                    rstd_pre=s["rstd_pre"])
    if op == "norm_bwd":
        return L.block_norm_backward(s["grad_out"], s["h"], s["summed"], s["rstd_post"], s["rstd_pre"], s["w_post"],
                                     s["w_pre"], gate=s["gate"], scale=s["scale"], grad_summed=s["grad_summed"],
                                     grad_h=s["grad_h"], grad_residual=s["grad_residual"], grad_gate=s["grad_gate"],
                                     grad_w_post=s["grad_w_post"], grad_w_pre=s["grad_w_pre"])
    if "optimizer" not in s:      # a training program keeps it next to the tensors
        s["optimizer"] = L.AdamW(_adamw_tensors(L, s), beta1=_BETA1, beta2=_BETA2, eps=_EPS, weight_decay=_DECAY)
    norm = s["optimizer"].step(s["step"], _LR, max_norm=s["max_norm"], seed=s["seed"])
    if s["moments"] == "8bit":
        s["optimizer"].moments(*s["moment_views"])
    return _adamw_outputs(s, norm)


def _adamw_tensors(L, s):
    tensors = []
    s["moment_views"] = [], []
    for at, n, decay in s["layout"]:
        here = slice(at, at + n)
        copy = None if s["copied"] is None else s["copied"][here]
        if s["moments"] == "float32":
            moments = {"m": s["m"][here], "v": s["v"][here]}
        else:
            b = slice(at // _BLOCK, (at + n + _BLOCK - 1) // _BLOCK)
            moments = {"m": s["m_codes"][here], "v": s["v_codes"][here], "m_scale": s["m_scale"][b],
                       "v_scale": s["v_scale"][b]}
            s["moment_views"][0].append(s["m"][here])
            s["moment_views"][1].append(s["v"][here])
        tensors.append(L.AdamWTensor(s["param"][here], s["gradient"][here], copy=copy, decay=decay, **moments))
    return tensors


def _adamw_outputs(s, norm):
    return {"norm": norm, "param": s["param"], "copy": s["copied"], "m": s["m"], "v": s["v"]}


def _plain(s):
    op = s["op"]
    if op == "loss":
        return _plain_loss(s)
    if op == "loss_bwd":
        x, table = s["x"].float(), s["table"].float()
        grad = torch.exp(x @ table.t() - s["lse"][:, None])
        target = s["target"].long()
        grad[torch.arange(len(target), device="cuda"), target.clamp(min=0)] -= 1.0
        grad *= torch.where(target >= 0, s["row_weight"], 0.0)[:, None]
        s["grad_x"].copy_(grad @ table)
        s["grad_table"].copy_(grad.t() @ x)
        return s["grad_x"], s["grad_table"]
    if op == "norm_fwd":
        return _plain_norm(s)
    if op == "norm_bwd":
        return _plain_norm_backward(s)
    return _plain_adamw(s)


def _plain_loss(s):
    logits = s["x"].float() @ s["table"].float().t()
    top = logits.max(1).values
    target = s["target"].long()
    chosen = logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
    s["lse"].copy_(top + torch.log(torch.exp(logits - top[:, None]).sum(1)))
    s["loss"].copy_(torch.where(target >= 0, s["row_weight"] * (s["lse"] - chosen), 0.0))
    return s["loss"], s["lse"]


def _plain_norm(s):
    dt = s["h"].dtype
    h, cols = s["h"].float(), s["h"].shape[1]
    rstd_post = torch.rsqrt((h * h).sum(1) / cols + _EPS_NORM)
    z = h * rstd_post[:, None] * s["w_post"].float() * s["scale"]
    if s["gate"] is not None:
        z = z / (1.0 + torch.exp(-s["gate"].float()))
    x = s["residual"].float() + z
    rstd_pre = torch.rsqrt((x * x).sum(1) / cols + _EPS_NORM)
    y = x * rstd_pre[:, None] * s["w_pre"].float()
    return y.to(dt), x.to(dt), rstd_post, rstd_pre


def _plain_norm_backward(s):
    dt = s["h"].dtype
    cols = s["h"].shape[1]
    dy, xhat = s["grad_out"].float(), s["summed"].float() * s["rstd_pre"][:, None]
    hhat = s["h"].float() * s["rstd_post"][:, None]
    g = dy * s["w_pre"].float()
    dx = s["rstd_pre"][:, None] * (g - xhat * ((g * xhat).sum(1) / cols)[:, None]) + s["grad_summed"].float()
    dz, grad_gate = dx * s["scale"], None
    if s["gate"] is not None:
        open_ = 1.0 / (1.0 + torch.exp(-s["gate"].float()))
        grad_gate = (dz * hhat * s["w_post"].float() * open_ * (1.0 - open_)).to(dt)
        dz = dz * open_
    g2 = dz * s["w_post"].float()
    dh = s["rstd_post"][:, None] * (g2 - hhat * ((g2 * hhat).sum(1) / cols)[:, None])
    return dh.to(dt), dx.to(dt), grad_gate, (dz * hhat).sum(0), (dy * xhat).sum(0)


def _plain_adamw(s):
    g = s["gradient"].float()
    norm = None
    if s["max_norm"] is not None:      # long sums, in 64 bits
        norm = torch.sqrt(s["gradient"].double().square_().sum())
        g = g * torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0).float()
        norm = norm.float()
    if s["moments"] == "float32":
        m, v = s["m"], s["v"]
    else:
        m = _decoded(s["m_codes"].float(), s["m_scale"])
        v = _decoded(s["v_codes"].float(), s["v_scale"]).square_()
    m.mul_(_BETA1).add_(g * (1.0 - _BETA1))
    v.mul_(_BETA2).add_((g * (1.0 - _BETA2)).mul_(g))
    del g
    root = torch.sqrt(v)
    update = m / (root * (1.0 / math.sqrt(1.0 - _BETA2 ** s["step"])) + _EPS)
    s["param"][:s["decayed"]] *= 1.0 - _LR * _DECAY
    s["param"] -= update * (_LR / (1.0 - _BETA1 ** s["step"]))
    if s["copied"] is not None:
        s["copied"].copy_(s["param"])
    if s["moments"] == "8bit":
        del update
        place = s["first"][:, None] + torch.arange(_BLOCK, device="cuda")
        bits = _scramble(place ^ s["keys"][:, None])
        del place
        s["m_codes"].copy_(_coded(m, s["m_scale"], _TOP_M, bits >> 16))
        s["v_codes"].copy_(_coded(root, s["v_scale"], _TOP_V, bits & 0xFFFF))
        s["m"].copy_(_decoded(s["m_codes"].float(), s["m_scale"]))
        s["v"].copy_(_decoded(s["v_codes"].float(), s["v_scale"]).square_())
    return _adamw_outputs(s, norm)


def _decoded(codes, scale):
    """A code q stands for sign(q) q^2 times its block's scale."""
    return (codes * codes.abs()).view(-1, _BLOCK).mul_(scale[:, None]).view(-1)


def _coded(x, scale, top, bits):
    """The codes of x, signed; writes the blocks' scales.  Between two codes
    the random number decides, such that the mean of the decoded values is x."""
    x = x.view(-1, _BLOCK)
    most = x.abs().max(1).values
    scale.copy_(most * (1.0 / top ** 2))
    y = x.abs() * torch.where(most > 1e-30, torch.full_like(most, top ** 2) / most, 0.0)[:, None]
    y.clamp_(max=float(top ** 2))
    low = torch.floor(torch.sqrt(y))
    low -= (low * low > y).float()
    low += ((low + 1.0) * (low + 1.0) <= y).float()
    up = (y - low * low) > (bits.float() * (1.0 / 65536.0)) * (2.0 * low + 1.0)
    return torch.copysign(low + up.float(), x).view(-1)


# --------------------------------------------------------------------------
# In 64 bits, from the definitions
# --------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("loss"):
        return _exact_loss(s)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    return _exact_norm(s)


def _exact_loss(s):
    n, step = s["x"].shape[0], 1024
    table = s["table"].double()
    target, valid = s["target"].long(), s["target"] >= 0
    weight = s["row_weight"].double() * valid
    loss, lse = [], []
    grad_x, grad_table = [], torch.zeros(table.shape, dtype=torch.float64, device="cuda")
    for r in range(0, n, step):
        x = s["x"][r:r + step].double()
        logits = torch.mm(x, table.t())
        hit = torch.zeros_like(logits)
        hit.scatter_(1, target[r:r + step].clamp(min=0)[:, None], 1.0)
        if s["op"] == "loss":
            lse.append(torch.logsumexp(logits, 1))
            loss.append(weight[r:r + step] * (lse[-1] - (logits * hit).sum(1)))
        else:
            d = (torch.exp(logits - s["lse"][r:r + step].double()[:, None]) - hit) * weight[r:r + step][:, None]
            grad_x.append(torch.mm(d, table))
            grad_table.addmm_(d.t(), x)
    return (torch.cat(loss), torch.cat(lse)) if s["op"] == "loss" else (torch.cat(grad_x), grad_table)


def _exact_norm(s):
    h, w1, w2 = s["h"].double(), s["w_post"].double(), s["w_pre"].double()
    gate = torch.ones_like(h) if s["gate"] is None else torch.sigmoid(s["gate"].double())
    if s["op"] == "norm_fwd":
        r1 = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + _EPS_NORM)
        x = s["residual"].double() + s["scale"] * gate * (h * r1 * w1)
        r2 = 1.0 / torch.sqrt(x.square().mean(1, keepdim=True) + _EPS_NORM)
        return x * r2 * w2, x, r1[:, 0], r2[:, 0]
    r1, r2 = s["rstd_post"].double()[:, None], s["rstd_pre"].double()[:, None]
    x, dy = s["summed"].double(), s["grad_out"].double()
    n = x.shape[1]
    # d/dx of y_j = x_j r w_j with dr/dx_i = -r^3 x_i / n, likewise for h.
    dx = s["grad_summed"].double() + r2 * w2 * dy - x * r2 ** 3 / n * (dy * w2 * x).sum(1, keepdim=True)
    normed = h * r1
    d_normed = dx * s["scale"] * gate * w1
    dh = r1 * d_normed - h * r1 ** 3 / n * (d_normed * h).sum(1, keepdim=True)
    d_gate = None if s["gate"] is None else dx * s["scale"] * normed * w1 * gate * (1.0 - gate)
    return dh, dx, d_gate, (dx * s["scale"] * gate * normed).sum(0), (dy * x * r2).sum(0)


def _exact_adamw(s):
    g = s["gradient"].double()
    norm = None
    if s["max_norm"] is not None:
        norm = torch.linalg.vector_norm(g)
        g = g * min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    if s["moments"] == "float32":
        m, v = s["m"].double(), s["v"].double()
    else:
        q = s["m_codes"].double().view(-1, _BLOCK)
        m = (torch.sign(q) * q ** 2 * s["m_scale"].double()[:, None]).view(-1)
        q = s["v_codes"].double().view(-1, _BLOCK)
        v = ((q ** 2 * s["v_scale"].double()[:, None]) ** 2).view(-1)
    m = _BETA1 * m + (1.0 - _BETA1) * g
    v = _BETA2 * v + (1.0 - _BETA2) * g ** 2
    del g
    p = s["param"].double()
    p[:s["decayed"]] -= _LR * _DECAY * p[:s["decayed"]]
    m_hat, v_hat = m / (1.0 - _BETA1 ** s["step"]), v / (1.0 - _BETA2 ** s["step"])
    p -= _LR * m_hat / (torch.sqrt(v_hat) + _EPS)
    del m_hat, v_hat
    if s["moments"] == "8bit":
        # Which of two codes a value gets can hang on the last bit of 32-bit
        # arithmetic, and one such value in a hundred thousand is more than
        # 32-bit values may be off: they have no value in 64 bits.
        m = v = None
    return {"norm": norm, "param": p, "copy": None if s["copied"] is None else p, "m": m, "v": v}

