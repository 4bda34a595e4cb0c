"""Plain implementations of the language model operators in 64 bits, with the
bounds that rounding gives their 32-bit results.

U is half a step of float32, relative.  A result's bound counts the roundings on
the way to it, in units of U times the sum of the absolute values that it is made
of, plus half a step of its own type."""

import numpy as np
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, want, units, size, name=""):
    """|got - want| <= units * U * size + half a step of got's type (of its smallest
    number where it is subnormal); NaN and infinities in the same places."""
    g, want = got.detach().double().cpu(), want.double().cpu()
    size = torch.as_tensor(size, dtype=torch.float64).cpu()
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(g)), name
    err = (g - want).abs()
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    tol = units * U * size + half_step(got.dtype) * want.abs() + tiny
    bad = (err > tol) & fine
    assert not bool(bad.any()), (name, int(bad.sum()), float((err / tol)[fine].max()))


# ---- block norm -------------------------------------------------------------


def norm_forward(h, residual, w1, w2, gate, scale, eps):
    """(y, summed, r1, r2) and the sizes of y and summed."""
    h, residual, w1, w2 = (t.double() for t in (h, residual, w1, w2))
    opened = torch.ones_like(h) if gate is None else torch.sigmoid(gate.double())
    r1 = 1 / torch.sqrt((h * h).mean(-1) + eps)
    z = scale * opened * h * r1[..., None] * w1
    x = residual + z
    r2 = 1 / torch.sqrt((x * x).mean(-1) + eps)
    y = x * r2[..., None] * w2
    size = residual.abs() + z.abs()
    return (y, x, r1, r2), (size * r2[..., None] * w2.abs(), size)


def norm_backward(dy, h, x, r1, r2, w1, w2, gate, scale, ds):
    """(dh, dx, dgate or None, dw1, dw2) and their sizes, from the formulas."""
    dy, h, x, r1, r2, w1, w2 = (t.double() for t in (dy, h, x, r1, r2, w1, w2))
    opened = torch.ones_like(h) if gate is None else torch.sigmoid(gate.double())
    r1, r2 = r1[..., None], r2[..., None]
    xhat, hhat, g = x * r2, h * r1, dy * w2
    dx = r2 * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    sx = r2 * (g.abs() + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True))
    if ds is not None:
        dx, sx = dx + ds.double(), sx + ds.double().abs()
    dz, sz = scale * opened * dx, abs(scale) * opened * sx
    q, sq = dz * w1, sz * w1.abs()
    dh = r1 * (q - hhat * (q * hhat).mean(-1, keepdim=True))
    sh = r1 * (sq + hhat.abs() * (sq * hhat.abs()).mean(-1, keepdim=True))
    dgate = None if gate is None else q * hhat * (1 - opened)
    sgate = None if gate is None else sq * hhat.abs() * (1 - opened)
    cols = h.shape[-1]
    total = lambda t: t.reshape(-1, cols).sum(0)   # noqa: E731
    return ((dh, dx, dgate, total(dz * hhat), total(dy * xhat)),
            (sh, sx, sgate, total(sz * hhat.abs()), total((dy * xhat).abs())))


# ---- linear cross entropy -----------------------------------------------------


def ce_forward(x, w, target, row_weight):
    """(loss, lse), and for each row the sum |x| |w| of its largest class."""
    z = x.double() @ w.double().t()
    size = (x.double().abs() @ w.double().abs().t()).max(-1).values
    lse = torch.logsumexp(z, -1)
    t = target.long()
    live = (t >= 0) & (t < w.shape[0])
    weight = torch.ones_like(lse) if row_weight is None else row_weight.double()
    live = live & (weight != 0)
    chosen = z.gather(-1, t.clamp(0, w.shape[0] - 1)[..., None])[..., 0]
    return torch.where(live, weight * (lse - chosen), 0.0), lse, size


def ce_backward(x, w, target, lse, row_weight):
    """(dx, dw, G): from the lse given."""
    z = x.double() @ w.double().t()
    t = target.long()
    weight = torch.ones(len(t), dtype=torch.float64, device=x.device) if row_weight is None else row_weight.double()
    live = (t >= 0) & (t < w.shape[0]) & (weight != 0)
    g = torch.exp(z - lse.double()[:, None])
    g[torch.arange(len(t), device=x.device), t.clamp(0, w.shape[0] - 1)] -= 1
    g = torch.where(live[:, None], g * weight[:, None], 0.0)
    xs = torch.where(live[:, None], x.double(), 0.0)
    return g @ w.double(), g.t() @ xs, g


# ---- AdamW --------------------------------------------------------------------

BLOCK = 256


def mix(h):
    """The final mixing of MurmurHash3 (32 bits) of uint64 arrays."""
    m = np.uint64(0xFFFFFFFF)
    h = h ^ (h >> np.uint64(16))
    h = h * np.uint64(0x85EBCA6B) & m
    h = h ^ (h >> np.uint64(13))
    h = h * np.uint64(0xC2B2AE35) & m
    return h ^ (h >> np.uint64(16))


def decode(codes, scale, square):
    """float32 values of codes (each step rounded), numpy."""
    q = codes.astype(np.float32)
    per = np.repeat(scale.astype(np.float32), BLOCK)[:len(q)]
    v = q * np.abs(q) * per
    return v * v if square else v


def encode(x, top, bits):
    """(codes, scales) of float32 x, in float32 arithmetic as documented."""
    n = len(x)
    blocks = -(-n // BLOCK)
    full = np.zeros(blocks * BLOCK, np.float32)
    full[:n] = x
    most = np.abs(full).reshape(blocks, BLOCK).max(1)
    scale = most * np.float32(1.0 / top ** 2)
    inv = np.where(most > 1e-30, np.float32(top ** 2) / np.maximum(most, np.float32(1e-38)), np.float32(0)).astype(np.float32)
    y = np.minimum(np.abs(x) * np.repeat(inv, BLOCK)[:n], np.float32(top ** 2)).astype(np.float32)
    low = np.floor(np.sqrt(y.astype(np.float64))).astype(np.float32)
    low -= low * low > y
    low += (low + 1) * (low + 1) <= y
    up = (y - low * low) > (bits.astype(np.float32) * np.float32(2.0 ** -16)) * (2 * low + 1)
    return np.copysign(low + up, x).astype(np.int64), scale


def adamw(p, g, m, v, t, lr, b1, b2, eps, wd, decay, clip=np.float32(1)):
    """One step in float32 arithmetic, each operation rounded: (p, m, root, v)."""
    f = np.float32
    g = g.astype(np.float32) * f(clip)
    m = m * f(b1) + g * f(1.0 - b1)
    v = v * f(b2) + (g * f(1.0 - b2)) * g
    root = np.sqrt(v)
    step = m / (root * f(1.0 / np.sqrt(1.0 - b2 ** t)) + f(eps))
    if decay:
        p = p * f(1.0 - lr * wd)
    return p - step * f(lr / (1.0 - b1 ** t)), m, root, v


def adamw_exact(p, g, m, v, t, lr, b1, b2, eps, wd, decay):
    """The same in 64 bits, from the definition."""
    p, g, m, v = (a.astype(np.float64) for a in (p, g, m, v))
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    p = p - lr * wd * p if decay else p
    return p - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps), m, v
