"""Plain float64 forms of the training operators, and bounds on what a
float32 computation of them may be off, for the tests of the kernels.

u = 2^-24 is float32's rounding unit, U[dtype] an output type's.  A sum of
terms t_i whose longest chain of additions is d long is off by at most
d * u * sum |t_i| (to first order); the kernels' chains are at most DEPTH
terms (a thread's own elements, 5 shuffles, 16 warps) for a row's sums."""

import math

import torch

F64 = torch.float64
u = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}   # below: no relative rounding
DEPTH = 64


def check(got, want, bound, what):
    """|got - want| <= bound wherever want is finite; the same elsewhere."""
    got, want = got.to(F64), want.to(F64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what + ": infinities differ"
    off = (got - want).abs()[fine]
    b = bound.to(F64).expand(want.shape)[fine]
    bad = ~(off <= b)
    assert not bad.any(), "%s: %d of %d off by more than the bound; worst %.3g against %.3g" % (
        what, int(bad.sum()), bad.numel(), float(off[bad].max()), float(b[bad][off[bad].argmax()]))


def rounded(want, dtype):
    return U[dtype] * want.abs() + TINY[dtype]


# ---- embedding -----------------------------------------------------------------


def embed_backward(grad_out, index, rows, scale):
    """(gradient, bound): the sum of a row's terms, each exact in float32, in
    a chain of at most its own length, then the scale."""
    real = (index >= 0) & (index < rows)
    g, i = grad_out.to(F64)[real], index.long()[real]
    cols = grad_out.shape[1]
    dev = grad_out.device
    out = torch.zeros(rows, cols, dtype=F64, device=dev).index_add_(0, i, g)
    mag = torch.zeros(rows, cols, dtype=F64, device=dev).index_add_(0, i, g.abs())
    count = torch.zeros(rows, dtype=F64, device=dev).index_add_(0, i, torch.ones_like(i, dtype=F64))
    return out * scale, (count[:, None] + 2) * u * mag * abs(scale) * 1.01


# ---- layer norm ------------------------------------------------------------------


def norm_forward(x, weight, bias, eps, residual=None):
    s = x.to(F64) if residual is None else x.to(F64) + residual.to(F64)
    mean = s.mean(1)
    var = ((s - mean[:, None]) ** 2).mean(1)
    rstd = 1.0 / torch.sqrt(var + eps)
    y = (s - mean[:, None]) * rstd[:, None] * weight.to(F64)
    if bias is not None:
        y = y + bias.to(F64)
    return y, s, mean, rstd


def norm_forward_bounds(s, mean, rstd, y, weight, bias, dtype):
    """Bounds of (y, summed, mean, rstd).  The mean is off by d = DEPTH u
    mean|s|; that and the sums' own rounding put the variance off by DEPTH u
    of itself plus d^2 plus the rounding of s - mean, rstd by half of that
    relatively."""
    mag = s.abs().mean(1)
    d = (DEPTH + 2) * u * mag
    var = 1.0 / rstd ** 2
    # s - mean: rounding of s itself (u |s|, a sum with a residual) and of the mean's error
    e = d + 2 * u * mag
    rel = (DEPTH + 8) * u + (2 * e * (s - mean[:, None]).abs().mean(1) + e ** 2) / var
    b_rstd = rel * rstd
    dev = (s - mean[:, None]).abs()
    w = weight.to(F64).abs()
    b_y = w * rstd[:, None] * (d[:, None] + 2 * u * s.abs()) + w * dev * rstd[:, None] * (rel[:, None] + 4 * u)
    b_y = b_y + 2 * u * (0 if bias is None else bias.to(F64).abs()) + rounded(y, dtype)
    return b_y * 1.01, rounded(s, dtype) * 1.01 + 2 * u * s.abs(), d, b_rstd * 1.01


def norm_backward(dy, x, mean, rstd, weight, dres=None):
    dy, xhat = dy.to(F64), (x.to(F64) - mean.to(F64)[:, None]) * rstd.to(F64)[:, None]
    g = dy * weight.to(F64)
    dx = rstd.to(F64)[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.to(F64)
    return dx, (dy * xhat).sum(0), dy.sum(0)


def norm_backward_bounds(dy, x, mean, rstd, weight, dx, dtype, dres=None):
    """Column sums: a thread's rows (no more than rows / 152 in a chain, or 1
    when there are fewer rows than blocks), 8 groups, 38 and 32 partial sums."""
    dy, xhat = dy.to(F64).abs(), ((x.to(F64) - mean.to(F64)[:, None]) * rstd.to(F64)[:, None]).abs()
    r = rstd.to(F64).abs()[:, None]
    g = dy * weight.to(F64).abs()
    k = (DEPTH + 8) * u
    b = r * k * (g + g.mean(1, keepdim=True) + xhat * (g * xhat).mean(1, keepdim=True)) + rounded(dx, dtype)
    if dres is not None:
        b = b + 2 * u * dres.to(F64).abs()
    chain = (84 + math.ceil(dy.shape[0] / 152)) * u
    return b * 1.01, chain * (dy * xhat).sum(0) * 1.01, chain * dy.sum(0) * 1.01


# ---- distillation ------------------------------------------------------------------


def _distribution(top_logits, top_index, cols, T):
    t = top_logits.to(F64)
    counts = (top_index >= 0) & (top_index < cols) & (t != -math.inf)
    t = torch.where(counts, t / T, -math.inf)
    some = counts.any(1)
    tm = torch.where(some, t.amax(1), torch.zeros_like(t[:, 0]))[:, None]
    logp = t - tm
    logp = logp - torch.log(torch.exp(logp).sum(1, keepdim=True))
    p = torch.where(counts, torch.exp(logp), 0.0)
    return counts, some, logp, p


def distill(logits, top_logits, top_index, T, row_weight=None):
    """(loss, grad) from the definition."""
    rows, cols = logits.shape
    w = torch.ones(rows, dtype=F64, device=logits.device) if row_weight is None else row_weight.to(F64)
    counts, some, logp, p = _distribution(top_logits, top_index, cols, T)
    z = logits.to(F64) / T
    z = z - z.amax(1, keepdim=True)          # log sum exp of values near 1e38 would swallow log(cols)
    logq = z - torch.logsumexp(z, 1, keepdim=True)
    index = torch.where(counts, top_index.long(), 0)
    terms = torch.where(counts & (p > 0), p * (logp - logq.gather(1, index)), 0.0)
    use = some & (w != 0)
    loss = torch.where(use, w * T * T * terms.sum(1), 0.0)
    grad = torch.exp(logq).scatter_add(1, index, -p) * (w * T)[:, None]
    return loss, torch.where(use[:, None], grad, 0.0)


def distill_bounds(logits, top_logits, top_index, T, grad, row_weight=None):
    """Bounds of (loss, grad).  An exponential ex2((z - m) log2e / T) has a
    relative error of 2^-22 (the instruction) plus 3 u |z - m| / T (its
    argument's roundings); s adds its chain (cols / 256 + 64 terms at most); the
    logarithms follow from those, and cost u of their own size."""
    rows, cols = logits.shape
    w = torch.ones(rows, dtype=F64, device=logits.device) if row_weight is None else row_weight.to(F64).abs()
    counts, some, logp, p = _distribution(top_logits, top_index, cols, T)
    z = logits.to(F64) / T
    m = z.amax(1, keepdim=True)
    a = torch.where(torch.isfinite(z - m), (m - z), 0.0)
    q = torch.softmax(z, 1)
    e_arg = 2.0 ** -22 + 4 * u * a                            # of one exponential
    e_s = (q * e_arg).sum(1, keepdim=True) + (cols / 256 + 64) * u   # of s
    e_q = e_arg + e_s + 4 * u
    tmax = torch.where(counts, top_logits.to(F64) / T, -math.inf).amax(1, keepdim=True)
    ta = torch.where(counts, tmax - top_logits.to(F64) / T, 0.0)
    e_t = 2.0 ** -22 + 4 * u * ta
    e_ps = (p * e_t).sum(1, keepdim=True) + 96 * u
    e_p = e_t + e_ps + 4 * u
    index = torch.where(counts, top_index.long(), 0)
    pd = torch.zeros_like(z).scatter_add_(1, index, p * e_p)
    b_grad = (w * T)[:, None] * (q * e_q + pd + 4 * u * (q + torch.zeros_like(z).scatter_add_(1, index, p)))
    logs = torch.logsumexp(z - m, 1, keepdim=True)
    za = torch.gather(a, 1, index)
    logp = torch.where(counts, logp, 0.0)
    logq = -(za + logs)
    e_term = e_ps + e_s + 4 * u * (ta + (ta + logp).abs() + za + logs.abs()) + (e_p + DEPTH * u) * (logp - logq).abs()
    b_loss = w * T * T * (p * e_term).sum(1)
    return b_loss * 1.01 + 1e-30, b_grad * 1.01
