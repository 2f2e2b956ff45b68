"""Plain 64-bit forms of the heads' norm with rotation, its gradients and the MXFP4 cache, and the error bounds
of their fp32 kernels (test infrastructure; torch float64 on whatever device its arguments are).

Bounds, with u = 2^-24. A head's sum has chains of at most 16 terms in a lane and a tree of 6: 24 u of
the sum of absolute values. The square root's reciprocal is then off by (24 + 2) u / 2 and its own 2 u: 15 u of itself,
a normed channel by 17 u. An angle is off by 2^-50 of itself (the frequency over 2 pi, the product and the
difference, in 64 bits), then its fraction of a turn is rounded to fp32: pi u; sine and cosine are good to 4 u and
multiplied by the amplitude: 9 u in all. A rotated channel a cos t - b sin t adds two products and a sum: 3 u of
(|a| + |b|) amplitude.
"""
import math

import torch

U = 2.0 ** -24
TURN = 12 * U  # of (|a| + |b|) amplitude, for exact a and b


def angles(positions, freq, axis_pairs, amplitude):
    """(cos, sin, bound of both) [m][1][pairs] times the amplitude."""
    p = positions.double().reshape(positions.shape[0], -1)
    t = torch.cat([p[:, i:i + 1].expand(-1, n) for i, n in enumerate(axis_pairs)], 1) * freq
    off = t.abs() * 2.0 ** -50
    return (torch.cos(t)[:, None] * amplitude, torch.sin(t)[:, None] * amplitude, off[:, None] * abs(amplitude))


def pairs_of(x, half, inter):
    r = 2 * half
    return (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., :half], x[..., half:r])


def joined(a, b, rest, inter):
    return torch.cat((torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1), rest), -1)


def turn(x, tol, rope, back=False):
    """x turned, with the bound of the result for x off by tol; rope None: as they are."""
    if rope is None or rope["freq"].numel() == 0:
        return x, tol
    n, inter = rope["freq"].numel(), rope.get("inter", False)
    c, s, off = angles(rope["positions"], rope["freq"], rope.get("axis_pairs", (n,)), rope.get("amplitude", 1.0))
    s = -s if back else s
    amp = abs(rope.get("amplitude", 1.0))
    a, b = pairs_of(x, n, inter)
    ta, tb = pairs_of(tol, n, inter)
    size = a.abs() + b.abs()
    # |cos| and |sin| are at most 1
    t = (ta + tb) * amp + size * (TURN * amp + off)
    y = joined(a * c - b * s, b * c + a * s, x[..., 2 * n:], inter)
    return y, joined(t, t, tol[..., 2 * n:], inter)


def weights(w_q, w_k, q, heads, d, device):
    one = torch.ones(d, dtype=torch.float64, device=device)
    return torch.stack([(one if w is None else w.double()) for w in [w_q] * q + [w_k] * (heads - q)] or
                       [one])[:heads]


def forward(x, w_q, w_k, q, eps, rope, norm=True):
    """(y, its bound before the rounding)"""
    x = x.double()
    if not norm:
        return turn(x, 0 * x, rope)
    rs = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = x * rs * weights(w_q, w_k, q, x.shape[1], x.shape[2], x.device)
    return turn(n, 17 * U * n.abs(), rope)


def backward(dy, x, w_q, w_k, q, eps, rope, norm=True):
    """((dx, dweight_q, dweight_k), their bounds before the rounding)"""
    dy = dy.double()
    e, e_tol = turn(dy, 0 * dy, rope, back=True)
    if not norm:
        return (e, None, None), (e_tol, None, None)
    x = x.double()
    m, heads, d = x.shape
    w = weights(w_q, w_k, q, heads, d, x.device)
    rs = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    h = x * rs
    g = e * w
    c = (g * h).mean(-1, keepdim=True)
    dx = rs * (g - h * c)
    # sum of (x w) e: 24 u and 2 u of its terms and e's own bound; times s (15 u) and 1 / d (3 u)
    mag = (h * g).abs().mean(-1, keepdim=True)
    c_tol = 44 * U * mag + (h * w).abs().mul(e_tol).mean(-1, keepdim=True)
    # h is off by 16 u of itself, the products and the difference by 3 u, all times s off by 15 u
    dx_tol = rs * (e_tol * w.abs() + 3 * U * g.abs() + h.abs() * (c_tol + 19 * U * c.abs())) + 17 * U * dx.abs()
    parts = max(1, min(256, (m + 3) // 4))
    chain = heads * -(-m // parts) + 64  # a lane's rows, the lanes, waves and parts
    s = e * h
    s_tol = (h.abs() * (e_tol + 17 * U * e.abs()) + chain * U * s.abs())
    return ((dx, s[:, :q].sum((0, 1)), s[:, q:].sum((0, 1))),
            (dx_tol, s_tol[:, :q].sum((0, 1)), s_tol[:, q:].sum((0, 1))))


LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
BORDERS = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)


def exponent(top):
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127)
    return torch.where(top > 0, e, -127)


def assert_codes_near(codes, scales, y, tol, what=""):
    """codes [..][d/2], scales [..][d/32] are a quantization of values within tol of y: the scale that of a maximum
    within its bound, each magnitude's index between those of |y| - tol and |y| + tol (ties may go either way),
    the sign y's unless |y| <= tol."""
    blocks = y.unflatten(-1, (-1, 32))
    t = tol.unflatten(-1, (-1, 32))
    mag = blocks.abs()
    e = scales.int() - 127
    lo, hi = exponent((mag - t).clamp(min=0).amax(-1)), exponent((mag + t).amax(-1))
    assert bool(((e >= lo) & (e <= hi)).all()), what + ": scales"
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, 32)).int()
    borders = BORDERS.to(y.device)
    step = torch.ldexp(torch.ones_like(mag), -e[..., None])
    least = torch.bucketize(((mag - t).clamp(min=0) * step).contiguous(), borders)               # border itself: below
    most = torch.bucketize(((mag + t) * step).contiguous(), borders, right=True)  # border itself: above
    index = code & 7
    assert bool(((index >= least) & (index <= most)).all()), what + ": codes"
    sign = (code >> 3) == (blocks < 0).int()
    assert bool((sign | (mag <= t)).all()), what + ": signs"
