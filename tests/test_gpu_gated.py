"""The gated products against plain binary64 forms: every gate, both types, one
row to many, odd sizes, strides with NaN in the padding, split sums, 8 bits kept
and read."""
import sys

import pytest

from communication_compressed_optimizer_02_amd import binding as oba
from layer_common import (U, check_kept, close, encode64, gen, half, out_rows, rows, tiny, torch,
                          untouched)
from sublayer_common import GATES, UNIT, gate64, gate_bounds

pytestmark = pytest.mark.gpu
TWO = ("f16", "bf16")
# rows, in, hidden (forward); rows, out, hidden (gradient)
SHAPES = [(1, 1, 1), (1, 40, 72), (1, 1600, 6400), (3, 64, 64), (7, 33, 129), (16, 5000, 16),
          (33, 520, 200), (64, 4096, 100), (130, 200, 77), (128, 128, 128), (257, 72, 400),
          (515, 777, 1001), (2000, 1000, 24), (1500, 40, 3600), (700, 1100, 513),
          # results of many tiles: more tiles than CUs and fewer, sums of less than a step,
          # of whole steps and with a remainder
          (8200, 40, 1033), (2300, 777, 4000), (8200, 130, 1700), (4100, 200, 3300),
          (8193, 128, 1700), (8193, 192, 3400)]


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def products(x, w):
    """x w^T and how far a binary32 sum of it may be off."""
    a, b = x.double(), w.double()
    return a @ b.t(), (x.shape[1] + 2) * U * (a.abs() @ b.abs().t()) + 1e-30


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("r,i,h", SHAPES)
def test_gated_linear(r, i, h, gate):
    t = torch()
    dtype = TWO[(r + i + h + len(gate)) % 2]
    say(f"[gated] {r}x{i} -> {h} {dtype} {gate}")
    g = gen(r * 7 + i * 3 + h)
    x = rows(g, r, i, dtype, extra=8)
    w = rows(g, 2 * h, i, dtype, std=i ** -0.5)
    bias = t.randn(2 * h + 1, generator=g, device="cuda")[1:] if len(gate) % 2 else None
    y, buf = out_rows(r, h, dtype)
    kept = [oba.act8_buffers(r, h) for _ in range(3)]
    ws = oba.gated_linear_workspace(r, i, h)
    oba.gated_linear(x, w, y, ws, bias=bias, gate=gate, qp=kept[0][0], ep=kept[0][1],
                     qu=kept[1][0], eu=kept[1][1], q=kept[2][0], e=kept[2][1])
    t.cuda.synchronize()
    pu, err = products(x, w)
    if bias is not None:
        pu = pu + bias.double()
        err = err + U * (pu.abs() + bias.double().abs())
    p, u, ep, eu = pu[:, :h], pu[:, h:], err[:, :h], err[:, h:]
    f, _ = gate64(p, gate)
    # |f'| < 1.13 for every gate
    ef = 1.13 * ep + gate_bounds(p, gate)[0]
    ref = f * u
    ey = ef * u.abs() + eu * (f.abs() + ef) + UNIT * ref.abs()
    close(y, ref, ey + (half(dtype) * (1 + 2 ** -7)) * ref.abs() + tiny(dtype) + 2.0 ** -120, "y")
    untouched(buf, h)
    check_kept(*kept[0], p, ep, "p")
    check_kept(*kept[1], u, eu, "u")
    q, e = oba.act8_buffers(r, h)
    oba.act8_encode(y, q, e)
    y2, _ = out_rows(r, h, dtype)
    oba.gated_linear(x, w, y2, ws, bias=bias, gate=gate)
    t.cuda.synchronize()
    assert t.equal(q, kept[2][0]) and t.equal(e, kept[2][1]), "y in 8 bits"
    assert t.equal(y, y2), "keeping in 8 bits changes the result"


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("r,o,h", SHAPES)
def test_gated_hidden_grad(r, o, h, gate):
    t = torch()
    dtype = TWO[(r + o + h + len(gate)) % 2]
    say(f"[gated grad] {r}x{o} -> {h} {dtype} {gate}")
    g = gen(r * 5 + o * 11 + h)
    dy = rows(g, r, o, dtype, extra=8)
    w = rows(g, o, h, dtype, std=o ** -0.5)
    qp, ep, p = encode64(rows(g, r, h, "f32", std=1.5))
    qu, eu, u = encode64(rows(g, r, h, "f32"))
    dpu, buf = out_rows(r, 2 * h, dtype)
    oba.gated_hidden_grad(dy, w, qp, ep, qu, eu, dpu, oba.gated_hidden_grad_workspace(r, h, o),
                          gate=gate)
    t.cuda.synchronize()
    d6, w6 = dy.double(), w.double()
    d, ed = d6 @ w6, (o + 2) * U * (d6.abs() @ w6.abs()) + 1e-30
    f, df = gate64(p, gate)
    ef, edf = gate_bounds(p, gate)
    for got, a, ea, what in ((dpu[:, :h], df * u, edf * u.abs(), "dp"), (dpu[:, h:], f, ef, "du")):
        ref = d * a
        err = ed * (a.abs() + ea) + d.abs() * ea + 2 * UNIT * ref.abs()
        close(got, ref, err + (half(dtype) * (1 + 2 ** -7)) * ref.abs() + tiny(dtype)
              + 2.0 ** -120, what)
    untouched(buf, 2 * h)


@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_gates_over_all_of_binary32(gate):
    """p is the bias alone.  Far from 0 the logistic function is 1, or 0 before
    binary32's range ends: silu's product is then off by less than 2^-110."""
    t = torch()
    for r in (1, 130):
        vals = [s * v for v in (0.0, 1e-30, 1e-3, 1.0, 20.0, 60.0, 87.0, 90.0, 1e3, 1e10, 1e30,
                                3e38) for s in (1.0, -1.0)]
        h = 32 * len(vals)
        p = t.tensor(vals, device="cuda").repeat_interleave(32)
        bias = t.cat([p, t.ones_like(p)])
        x = t.zeros((r, 8), device="cuda", dtype=t.bfloat16)
        w = t.zeros((2 * h, 8), device="cuda", dtype=t.bfloat16)
        y = t.empty((r, h), device="cuda", dtype=t.bfloat16)
        k = [oba.act8_buffers(r, h) for _ in range(2)]
        oba.gated_linear(x, w, y, oba.gated_linear_workspace(r, 8, h), bias=bias, gate=gate,
                         qp=k[0][0], ep=k[0][1], qu=k[1][0], eu=k[1][1])
        t.cuda.synchronize()
        p6 = p.double().expand(r, h)
        ref = gate64(p6, gate)[0]
        close(y, ref, gate_bounds(p6, gate)[0] + half("bf16") * (1 + 2 ** -7) * ref.abs()
              + 2.0 ** -110, "f")
        dy = t.ones((r, 8), device="cuda", dtype=t.bfloat16)
        w2 = t.zeros((8, h), device="cuda", dtype=t.bfloat16)
        w2[0] = 1.0
        dpu = t.empty((r, 2 * h), device="cuda", dtype=t.bfloat16)
        oba.gated_hidden_grad(dy, w2, *k[0], *k[1], dpu, oba.gated_hidden_grad_workspace(r, h, 8),
                              gate=gate)
        t.cuda.synchronize()
        from layer_common import decode64
        p8 = decode64(*k[0], h)
        f, df = gate64(p8, gate)
        ef, edf = gate_bounds(p8, gate)
        hb = half("bf16") * (1 + 2 ** -7)
        close(dpu[:, :h], df, edf + hb * df.abs() + 2.0 ** -110, "dp")
        close(dpu[:, h:], f, ef + hb * f.abs() + 2.0 ** -110, "du")


def test_infinities_and_nan_stay_where_they_belong():
    """An infinity in a row of x reaches that row alone; kept groups with one have
    the byte 255 and stand for NaN in the gradient."""
    t = torch()
    for r in (5, 200):
        g = gen(r)
        i, h = 96, 130
        x, w = rows(g, r, i, "bf16"), rows(g, 2 * h, i, "bf16", std=0.1)
        ws = oba.gated_linear_workspace(r, i, h)

        def run(x):
            y = out_rows(r, h, "bf16")[0]
            k = [oba.act8_buffers(r, h) for _ in range(3)]
            oba.gated_linear(x, w, y, ws, gate="silu", qp=k[0][0], ep=k[0][1], qu=k[1][0],
                             eu=k[1][1], q=k[2][0], e=k[2][1])
            t.cuda.synchronize()
            return y, k

        y0, _ = run(x)
        x[3, 50] = float("inf")
        y1, k = run(x)
        keep = t.arange(r, device="cuda") != 3
        assert t.equal(y0[keep], y1[keep]) and bool((~t.isfinite(y1[3])).all())
        assert bool((k[0][1][3] == 255).all()) and bool((k[1][1][3] == 255).all())
        dy, w2 = rows(g, r, 40, "bf16"), rows(g, 40, h, "bf16")
        dpu = out_rows(r, 2 * h, "bf16")[0]
        oba.gated_hidden_grad(dy, w2, *k[0], *k[1], dpu,
                              oba.gated_hidden_grad_workspace(r, h, 40))
        t.cuda.synchronize()
        assert bool(t.isnan(dpu[3]).all()) and bool(t.isfinite(dpu[keep]).all())


def test_no_rows_and_results_do_not_depend_on_the_workspace():
    t = torch()
    x = t.empty((0, 40), device="cuda", dtype=t.bfloat16)
    w = t.ones((48, 40), device="cuda", dtype=t.bfloat16)
    y = t.empty((0, 24), device="cuda", dtype=t.bfloat16)
    oba.gated_linear(x, w, y, None)
    q, e = oba.act8_buffers(0, 24)
    oba.gated_hidden_grad(x, t.ones((40, 24), device="cuda", dtype=t.bfloat16), q, e, q, e,
                          t.empty((0, 48), device="cuda", dtype=t.bfloat16), None)
    g = gen(1)
    x, w = rows(g, 100, 3000, "f16"), rows(g, 128, 3000, "f16", std=0.02)
    got = []
    for fill in (0, 255, 0x7F):
        ws = oba.gated_linear_workspace(100, 3000, 64)
        ws.fill_(fill)
        y = out_rows(100, 64, "f16")[0]
        oba.gated_linear(x, w, y, ws)
        t.cuda.synchronize()
        got.append(y)
    assert t.equal(got[0], got[1]) and t.equal(got[0], got[2])
