"""Plain binary64 forms of the gated feed-forward sub-layer's operators.
Tolerances count as layer_common's do."""
from __future__ import annotations

import math

import numpy as np

from layer_common import act64, act_grad64, torch

GATES = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid")
UNIT = 2.0 ** -24  # half a step of binary32


def philox(counter, key):
    """Philox4x32-10: four arrays of counter words and two key words to four
    arrays of words."""
    m = np.uint64(0xFFFFFFFF)
    s = np.uint64(32)
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k0, k1 = (int(v) for v in key)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s) ^ c[1] ^ np.uint64(k0), b & m, (a >> s) ^ c[3] ^ np.uint64(k1), a & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def factor(rows, cols, rate, seed, step, site, first_row=0):
    """[rows][cols] float64 numpy: 0 where dropped, else 65536 / (65536 - t)."""
    t = math.floor(rate * 65536 + 0.5)
    w = -(-cols // 8)
    i = np.arange(rows * w, dtype=np.uint64) + np.uint64(first_row * w)
    m = np.uint64(0xFFFFFFFF)
    full = lambda v: np.full(i.shape, v & 0xFFFFFFFF, dtype=np.uint64)  # noqa: E731
    words = philox([i & m, i >> np.uint64(32), full(site), full(step)],
                   [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF])
    bits = np.stack([(words[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF)
                     for j in range(8)], axis=1)
    keep = (bits >= np.uint64(t)).reshape(rows, w * 8)[:, :cols]
    return keep * (65536.0 / (65536 - t))


def factor_gpu(*a, **k):
    return torch().from_numpy(factor(*a, **k)).cuda()


def gate64(p, kind):
    """f(p) and f'(p)."""
    t = torch()
    if kind in ("silu", "sigmoid"):
        s, o = t.sigmoid(p), t.sigmoid(-p)
        return (p * s, s * (1 + p * o)) if kind == "silu" else (s, s * o)
    return act64(p, kind), act_grad64(p, kind)


def gate_bounds(p, kind):
    """How far f(p) and f'(p) may be off as they are evaluated.

    The logistic function: z = exp2(-log2(e) |p|) has a constant's and a product's
    rounding in its exponent (2 |p| of a unit), exp2 and the reciprocal are 2 units
    each, 1 + z and z t one each: (2 |p| + 6) units of s and of 1 - s.  silu' = s
    (1 + p (1 - s)) has s's error in all of it and (1 - s)'s in a part, and two
    more roundings.  GELU's Phi: (32 + 1.5 p^2) units (exponent 1.5 p^2, fit 15,
    exp2 and reciprocal 4, polynomial and products 10), exp(-p^2/2) (4 + 1.5 p^2).
    The tanh form's factor: (8 + 16 |u|) units where the exponential matters."""
    t = torch()
    f, d = gate64(p, kind)
    a = p.abs()
    if kind in ("silu", "sigmoid"):
        s, o, e = t.sigmoid(p), t.sigmoid(-p), (2 * a + 6) * UNIT
        if kind == "sigmoid":
            return e * f, (2 * e + UNIT) * d
        return (e + UNIT) * f.abs(), s * (e * (1 + a * o) + a * o * e + 2 * UNIT * (1 + a * o))
    if kind == "gelu":
        e = (33 + 1.5 * p * p) * UNIT
        phi = t.exp(-p * p / 2) / math.sqrt(2 * math.pi)
        cdf = 0.5 * t.erfc(-p / math.sqrt(2.0))
        return (e + UNIT) * f.abs(), e * (cdf + a * phi) + 2 * UNIT * d.abs()
    if kind == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (p + 0.044715 * p ** 3)
        s, o = t.sigmoid(2 * u), t.sigmoid(-2 * u)
        e = (10 + 16 * u.abs() * o) * UNIT
        slope = math.sqrt(2 / math.pi) * (2 + 6 * 0.044715 * p * p)
        # 1 - s is a difference from 1: off by a unit, and by s's error
        rest = a * slope * s * (o * (e + 8 * UNIT) + s * e + UNIT)
        return (e + UNIT) * f.abs(), s * e + rest + UNIT * d.abs()
    return t.zeros_like(p), t.zeros_like(p)


def norm_rows64(x, eta, kind):
    """Normalised rows and rstd (as a column)."""
    z = x - x.mean(1, keepdim=True) if kind == "layer" else x
    rstd = 1 / (z.square().mean(1, keepdim=True) + eta).sqrt()
    return z * rstd, rstd


def norm_rows_bound(x, ex, eta, kind):
    """Bounds of normalised rows (absolute) and of rstd (relative, a column) for
    rows off by ex.  Centred values have two roundings of their own size and the
    mean's 2^-48 of the largest value, and what the rows are off by, also through
    the mean; the mean square has 30 additions and products (up to 16 columns a
    lane, 6 exchanges), which a root halves, and what the centred values are off
    by; sum, root and quotient round once each."""
    h, rs = norm_rows64(x, eta, kind)
    z = h / rs
    ez = ex + 2 * UNIT * z.abs()
    if kind == "layer":
        ez = ez + ex.mean(1, keepdim=True) + 2.0 ** -48 * x.abs().amax(1, keepdim=True)
    # |root(z + ez) - root(z)| <= root(ez), root the root mean square
    rel = rs * ez.square().mean(1, keepdim=True).sqrt() + 20 * UNIT
    return (ez * rs) * (1 + rel) + h.abs() * (rel + UNIT), rel


def through64(a, h, rstd, kind):
    """A norm's input gradient from that of its normalised rows."""
    d = a - h * (a * h).mean(1, keepdim=True)
    if kind == "layer":
        d = d - a.mean(1, keepdim=True)
    return d * rstd


def through_bound(a, ea, h, rstd, kind):
    """For a off by ea: the sums have 16 columns a lane, 6 exchanges and 16 waves,
    38 additions and the products, each mean a quotient's rounding; the differences
    and products four more roundings of their operands."""
    m2 = (a * h).mean(1, keepdim=True)
    em2 = ((ea + 41 * UNIT * a.abs()) * h.abs()).mean(1, keepdim=True)
    e = ea + h.abs() * em2 + 4 * UNIT * (a.abs() + (h * m2).abs())
    if kind == "layer":
        e = e + (ea + 41 * UNIT * a.abs()).mean(1, keepdim=True) \
            + 4 * UNIT * a.mean(1, keepdim=True).abs()
    return rstd * e
