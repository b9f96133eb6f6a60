"""Layer norm of rows whose mean is far larger than their spread, and of
constant rows: what is normalised is centred on the mean to the accuracy of
the spread, not to that of the mean."""
import sys

import pytest

from communication_compressed_optimizer_02_amd import binding as oba
from layer_common import U, check_kept, close, dt, gen, half, norm64, out_rows, rows, torch

pytestmark = pytest.mark.gpu
ETA = 1e-5


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def forward(x, gamma, beta):
    t = torch()
    r, c = x.shape
    name = {t.float32: "f32", t.float16: "f16", t.bfloat16: "bf16"}[x.dtype]
    y, _ = out_rows(r, c, name)
    mean, rstd = t.empty(r, device="cuda"), t.empty(r, device="cuda")
    q, e = oba.act8_buffers(r, c)
    oba.layer_norm(x, gamma, beta, ETA, y, mean, rstd, q=q, e=e)
    t.cuda.synchronize()
    return y, mean, rstd, q, e


# one instance of the kernel each (columns of a wave, of 4 and of 8 waves)
@pytest.mark.parametrize("c", [40, 1000, 1600, 4090, 8000, 16384])
@pytest.mark.parametrize("at,std", [(1e3, 0.1), (1e3, 0.01), (1e4, 1.0), (-1e5, 1.0)])
def test_mean_far_from_zero(c, at, std):
    t = torch()
    r = 9
    say(f"[norm centre] {r}x{c} f32 mean {at} spread {std}")
    g = gen(int(abs(at)) + c)
    x = rows(g, r, c, "f32", std=std, extra=8)
    x += at
    gamma, beta = (t.randn(c, generator=g, device="cuda") for _ in range(2))
    y, mean, rstd, q, e = forward(x, gamma, beta)
    m, s, z = norm64(x, ETA)
    var, az = (z * z).mean(1), z.abs().mean(1)
    # a first mean from sums of 50 additions; the values less this mean, v,
    # each rounded once; their mean `off` from 50 additions of terms that are
    # as small as the spread and that error
    e1 = 50 * U * x.double().abs().amax(1)
    off = 52 * U * (az + e1)
    close(mean, m, off + half("f32") * m.abs(), "mean")
    ez = (2 * U * (z.abs() + e1[:, None])) + off[:, None]
    # the variance is the mean square of v less off^2
    ev = 55 * U * (var + e1 * e1) + 2 * e1 * off + U * e1 * e1
    es = s * (0.6 * ev / (var + ETA) + 3 * U)
    close(rstd, s, es, "rstd")
    h = z * s[:, None]
    eh = ez * s[:, None] + h.abs() * (es / s)[:, None] + 2 * U * h.abs()
    ref = h * gamma.double() + beta.double()
    close(y, ref, eh * gamma.double().abs() + 2 * U * ((h * gamma.double()).abs() + ref.abs()),
          "y")
    check_kept(q, e, h, eh, "xhat")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("c", [1, 33, 1000, 1600, 4090, 8192, 16001])
def test_constant_rows(c, dtype):
    """The first mean is a few units in the last place of the value off, the
    sum of that over the row is exact (7 and 14 bits), so xhat is 0."""
    t = torch()
    r = 12
    say(f"[norm centre] {r}x{c} {dtype} constant rows")
    g = gen(c)
    v = 1000.0 + 19000.0 * t.rand((r, 1), generator=g, device="cuda")
    x = rows(g, r, c, dtype, std=0.0)
    x += v.to(x.dtype)
    beta = t.randn(c, generator=g, device="cuda")
    y, mean, rstd, q, e = forward(x, t.randn(c, generator=g, device="cuda"), beta)
    assert t.equal(mean, x[:, 0].float()), "mean"
    assert t.equal(y, beta.to(dt(dtype)).expand(r, c)), "y"
    assert bool((q == 0).all()) and bool((e == 1).all()), "xhat"
    e1 = 50 * U * v.double()[:, 0]
    ev = 161 * U * e1 * e1  # as above, without a spread
    close(rstd, t.full_like(ev, ETA ** -0.5), ETA ** -0.5 * (0.6 * ev / ETA + 3 * U), "rstd")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("c", [7, 500, 1000, 1600, 4090, 8000, 16384])
def test_mean_near_zero_keeps_its_relative_accuracy(c, dtype):
    """Rows whose sum nearly cancels: each mean is its true value rounded once,
    up to what binary64 loses of the sum (2^-53 of the magnitudes for each of
    at most 16384 additions)."""
    t = torch()
    r = 40
    say(f"[norm centre] {r}x{c} {dtype} means near 0")
    g = gen(c + 1)
    x = rows(g, r, c, dtype, std=1.0)
    for k in range(3):  # takes the sum out of every row, up to the type's rounding
        left = x.double().sum(1)
        x[:, k] -= (left * (1 - 2.0 ** -9)).to(x.dtype)
    y, mean, rstd, q, e = forward(x, t.ones(c, device="cuda"), t.zeros(c, device="cuda"))
    m = x.double().sum(1) / c
    lost = 2.0 ** -53 * 16384 * x.double().abs().mean(1)
    close(mean, m, half("f32") * m.abs() * (1 + 2.0 ** -20) + lost, "mean")
