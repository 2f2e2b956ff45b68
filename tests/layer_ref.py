"""Plain 64-bit forms of the layer around the W4A4 product and the error bounds of its fp32 kernels
(test infrastructure; torch float64 on whatever device its arguments are).

Bounds. u = 2^-24 is the relative rounding of fp32. A sum of d terms of which a thread adds up
d / 64 at most, one after another, before a tree joins the threads is off by at most
L(d) u sum |terms| with L = d / 64 + 24. Rounding to the output type adds eps / 2 of the value.
"""
import math

import torch

U = 2.0 ** -24
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def L(d):
    return d / 64 + 24


def half_step(dtype, v):
    """A rounding of v to dtype is off by at most this (the smallest subnormal covers tiny v)."""
    f = torch.finfo(dtype)
    return v.abs() * (f.eps / 2) + f.smallest_normal * f.eps


# --- layer norm ------------------------------------------------------------------------------
def norm(x, w, b, eps):
    """(y, mean, rstd, bound of y before its rounding, bound of mean, relative bound of rstd)"""
    x = x.double()
    d = x.shape[1]
    w = torch.ones(d, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros(d, dtype=torch.float64, device=x.device) if b is None else b.double()
    mu = x.mean(1, keepdim=True)
    c = x - mu
    var = (c * c).mean(1, keepdim=True)
    rs = (var + eps).rsqrt()
    h = c * rs
    y = h * w + b
    spread = c.abs().mean(1, keepdim=True)
    # the first mean is off by L u mean |x|; the second pass corrects it, up to L u of what it sums,
    # and x minus the first mean is rounded
    first = L(d) * U * x.abs().mean(1, keepdim=True)
    around = spread + first
    mean_tol = U * mu.abs() + (L(d) + 2) * U * around
    rstd_tol = (L(d) + 8) * U * (1 + (first / (var + eps).sqrt()))
    h_tol = rs * ((L(d) + 2) * U * around + 3 * U * (c.abs() + first)) + h.abs() * (rstd_tol + 2 * U)
    y_tol = w.abs() * h_tol + 3 * U * ((h * w).abs() + b.abs())
    return y, mu[:, 0], rs[:, 0], y_tol, mean_tol[:, 0], rstd_tol[:, 0]


def norm_grad(dy, x, mean, rstd, w, parts_rows=64):
    """((dx, dw, db), their bounds before rounding), for the saved mean and rstd."""
    x, dy, mean, rstd = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    m, d = x.shape
    w = torch.ones(d, dtype=torch.float64, device=x.device) if w is None else w.double()
    h = (x - mean) * rstd
    g = dy * w
    a, b = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = rstd * (g - a - h * b)
    # h and g are off by 2 u and 1 u of themselves, their products by 4 u
    a_tol, b_tol = (L(d) + 3) * U * g.abs().mean(1, keepdim=True), (L(d) + 6) * U * (g * h).abs().mean(1, keepdim=True)
    dx_tol = rstd * (a_tol + h.abs() * b_tol + 6 * U * (g.abs() + a.abs() + (h * b).abs()))
    # a column: at most `rows` terms in one chain, then the partial sums of up to 512 parts
    rows = m / 16 + 512 + 24
    return (dx, (dy * h).sum(0), dy.sum(0)), (dx_tol, (rows + 4) * U * (dy * h).abs().sum(0),
                                              rows * U * dy.abs().sum(0))


# --- the quantized product and its epilogue --------------------------------------------------
def decode(codes, scales):
    """deq of codes [r][k/2], scales [r][k/32] in float64."""
    lv = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64, device=codes.device)
    v = torch.stack((lv[(codes & 15).long()], lv[(codes >> 4).long()]), -1).flatten(1)
    return v * torch.pow(2.0, scales.double() - 127).repeat_interleave(32, 1)


def unpack_scales(packed, rows, k):
    """The packed layout [k/256][rows][8] back as [rows][k/32]."""
    return packed.view(k // 256, rows, 2, 4).permute(1, 0, 3, 2).reshape(rows, k // 32)


def act(z, name):
    """(value, slope)"""
    one = torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, 0 * one), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if name == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (
            1 + 3 * 0.044715 * z * z)
    return z, one


def act_tol(z, name):
    """Bounds of the kernels' own error in the value and the slope at an exact z. The logistic's
    argument is off by 4 u of itself and x s(x) (1 - s(x)) <= 0.23, its exp2, sum and reciprocal
    by 1 ulp each: 8 u of |z| in the value. The slope adds (1 - s), off by 2 u absolute, times
    |z| and, for gelu_tanh, the inner slope c (1 + 0.134 z^2), c = 2 sqrt(2 / pi). gelu: erf to
    1.5e-7 (half of it in P) and the arithmetic around it, 6 u of P <= 1."""
    a = z.abs()
    if name in ("none", "relu"):
        return 0 * a, 0 * a
    if name == "silu":
        return 8 * U * a, 16 * U * (1 + a)
    if name == "gelu":
        return (0.75e-7 + 6 * U) * a, 0.75e-7 + 16 * U + 0 * a
    inner = 1.6 * (1 + 0.134 * a * a)
    return 8 * U * a, 16 * U * (1 + a * inner.clamp(max=60))


def linear(ca, sa, cw, sw, bias, name, residual):
    """(out, z, bound of out, bound of z), both bounds before the output's rounding."""
    A, W = decode(ca, sa), decode(cw, sw)
    z = A @ W.t()
    # the matrix instructions' sums, the bound of the plain product's tests; the bias and the
    # sum over a workgroup's waves are covered by u of each
    tol = 64 * U * (A.abs() @ W.abs().t())
    if bias is not None:
        z = z + bias.double()
        tol = tol + 2 * U * (z.abs() + bias.double().abs())
    o, slope = act(z, name)
    near = 1.2 * tol  # no slope here exceeds 1.13
    o_tol = near + act_tol(z, name)[0]
    if residual is not None:
        o = o + residual.double()
        o_tol = o_tol + U * o.abs()
    return o, z, o_tol + 2 * U * o.abs(), tol


def linear_grad(dout, z, name):
    """((dz, dbias), their bounds before rounding)"""
    dout, z = dout.double(), z.double()
    slope = act(z, name)[1]
    dz = dout * slope
    tol = dout.abs() * act_tol(z, name)[1] + 2 * U * dz.abs()
    rows = dz.shape[0] / 16 + 512 + 24
    return (dz, dz.sum(0)), (tol, tol.sum(0) + rows * U * dz.abs().sum(0))


# --- comparison ------------------------------------------------------------------------------
def assert_near(got, want, tol, what=""):
    """|got - want| <= tol + the rounding of want to got's type, elementwise."""
    d = (got.double() - want).abs()
    lim = tol + half_step(got.dtype, want.abs() + tol)
    bad = ~(d <= lim)
    assert not bool(bad.any()), "%s: %d of %d outside, worst %.3g x its bound at %s" % (
        what, int(bad.sum()), bad.numel(), float((d / lim).nan_to_num(nan=float("inf")).max()),
        torch.argwhere(bad)[0].tolist())
