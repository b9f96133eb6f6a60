"""Plain binary64 forms of the layer operators and the inputs of their tests.
Tolerances are sums of named terms: a rounding to a type is off by at most
half a step (finfo.eps / 2 of the value), a binary32 sum of k terms by at most
k * 2^-23 of the terms' magnitudes (2^-23 and not 2^-24: whichever way an
addition inside a matrix instruction rounds)."""
from __future__ import annotations

import math

GROUP = 32
U = 2.0 ** -23


def torch():
    import torch as t

    return t


def dt(name):
    t = torch()
    return {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}[name]


def half(name):
    """Half a step of a type, relative to the value."""
    return torch().finfo(dt(name)).eps / 2


def tiny(name):
    """Half the spacing of a type's subnormals."""
    return {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[name]


def gen(seed):
    g = torch().Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows(g, r, c, dtype, std=1.0, pad=float("nan"), extra=0):
    """[r][c] inside rows of a multiple of 8 elements whose rest is `pad`: what
    lies there must not matter."""
    t = torch()
    ld = (c + 7) // 8 * 8 + extra
    buf = t.full((r, ld), pad, device="cuda", dtype=dt(dtype))
    buf[:, :c] = (t.randn((r, c), generator=g, device="cuda") * std).to(dt(dtype))
    return buf[:, :c]


def out_rows(r, c, dtype, extra=8, fill=7.0):
    """(view, whole buffer) of an output whose padding must stay `fill`."""
    t = torch()
    buf = t.full((r, (c + 7) // 8 * 8 + extra), fill, device="cuda", dtype=dt(dtype))
    return buf[:, :c], buf


def untouched(buf, c, fill=7.0):
    assert bool((buf[:, c:] == fill).all()), "columns past the last were written"


def pow2(j):
    """2^j exactly, binary64, for integers -1000 < j < 1000 (pow is not exact)."""
    t = torch()
    return ((j.to(t.int64) + 1023) << 52).view(t.float64)


def encode64(x):
    """(q, e, values) of the 8-bit form, for finite x."""
    t = torch()
    x = x.double()
    r, c = x.shape
    p = t.zeros((r, -(-c // GROUP) * GROUP), dtype=t.float64, device=x.device)
    p[:, :c] = x
    p = p.view(r, -(-c // GROUP), GROUP)
    top = p.abs().amax(dim=2)
    k = t.frexp(top)[1] - 1
    j = t.where(top > 0, t.clamp(k - 6, min=-126), t.full_like(k, -126))
    s = pow2(j).unsqueeze(2)
    q = t.clamp(t.round(p / s), -127, 127)
    w = -(-c // GROUP) * GROUP
    return q.to(t.int8).view(r, w), (j + 127).to(t.uint8), (q * s).view(r, w)[:, :c]


def decode64(q, e, c):
    t = torch()
    s = pow2(e.to(t.int64) - 127).repeat_interleave(GROUP, dim=1)
    return (q.double() * s)[:, :c]


def check_kept(q, e, p, err, what):
    """(q, e) is the 8-bit form of some matrix within err of p."""
    t = torch()
    r, c = p.shape
    got = decode64(q, e, c)
    s = pow2(e.to(t.int64) - 127).repeat_interleave(GROUP, dim=1)[:, :c]
    top = (q.view(r, -1)[:, :c].abs() == 127)
    lim = t.where(top, s, 0.5 * s) + err
    assert bool(((got - p).abs() <= lim).all()), f"{what}: kept values off"
    pad = -(-c // GROUP) * GROUP
    pp = t.zeros((r, pad), dtype=t.float64, device=p.device)
    ee = t.zeros((r, pad), dtype=t.float64, device=p.device)
    pp[:, :c], ee[:, :c] = p.abs(), err
    m = pp.view(r, -1, GROUP).amax(2)
    ge = ee.view(r, -1, GROUP).amax(2)
    st = pow2(e.to(t.int64) - 127)
    assert bool(((m <= 128 * st + ge) & ((m >= 64 * st - ge) | (e == 1))).all()), \
        f"{what}: steps off"
    assert bool((q.view(r, -1)[:, c:] == 0).all()), f"{what}: integers past the last column"


def act64(p, kind):
    t = torch()
    if kind == "relu":
        return t.clamp(p, min=0)
    if kind == "gelu":
        return p * 0.5 * t.erfc(-p / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return p * t.sigmoid(math.sqrt(8 / math.pi) * (p + 0.044715 * p ** 3))
    return p


def act_grad64(p, kind):
    t = torch()
    if kind == "relu":
        return (p > 0).double()
    if kind == "gelu":
        return 0.5 * t.erfc(-p / math.sqrt(2.0)) + p * t.exp(-p * p / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        a = math.sqrt(8 / math.pi)
        s = t.sigmoid(a * (p + 0.044715 * p ** 3))
        return s + p * s * (1 - s) * a * (1 + 3 * 0.044715 * p * p)
    return t.ones_like(p)


def norm64(x, eta):
    x = x.double()
    mean = x.mean(1)
    z = x - mean[:, None]
    return mean, 1 / ((z * z).mean(1) + eta).sqrt(), z


def norm_grad64(n, dy, gamma, rstd, h, add):
    t = torch()
    dy = dy.double()
    a = dy * gamma.double()
    dx = rstd.double()[:, None] * (a - a.mean(1, keepdim=True)
                                   - h * (a * h).mean(1, keepdim=True))
    if add is not None:
        dx = dx + add.double()
    c = dy.shape[1]
    return dx, (dy * h).reshape(n, -1, c).sum(1), dy.reshape(n, -1, c).sum(1)


def close(got, ref, tol, what):
    t = torch()
    got = got.double()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        lim = tol[i] if isinstance(tol, t.Tensor) and tol.dim() else tol
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: "
                             f"{float(got[i])!r} for {float(ref[i])!r}, allowed {float(lim):.3e}")
