"""The activation functions and their derivatives over all of binary32's
range, and to their stated accuracy where results are small."""
import math
import sys

import pytest

from communication_compressed_optimizer_02_amd import binding as oba
from layer_common import act64, act_grad64, close, decode64, half, torch

pytestmark = pytest.mark.gpu
HUGE = [1e10, 3e18, 1.5e19, 5e19, 1e20, 1e25, 1e30, 3e38]


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("r", [1, 130])
def test_huge_finite_pre_activations(r, act):
    """Far from 0 the functions are p or 0, their derivatives 1 or 0."""
    t = torch()
    say(f"[act range] {r} rows {act}")
    p = t.tensor([s * v for v in HUGE for s in (1.0, -1.0)], device="cuda")
    c = 32 * p.numel()  # a group of 32 columns for every value
    p = p.repeat_interleave(32).expand(r, c).contiguous()
    x = t.zeros((r, 8), device="cuda", dtype=t.bfloat16)
    w = t.zeros((c, 8), device="cuda", dtype=t.bfloat16)
    y = t.empty((r, c), device="cuda", dtype=t.bfloat16)
    q, e = oba.act8_buffers(r, c)
    oba.linear(x, w, y, oba.linear_workspace(r, 8, c), bias=p[0], act=act, q=q, e=e)
    t.cuda.synchronize()
    ref = t.clamp(p.double(), min=0.0)
    close(y, ref, half("bf16") * ref, "act")
    p8 = decode64(q, e, c)
    assert bool(((p8 - p.double()).abs() <= 2.0 ** -6 * p.double().abs()).all())
    dy = t.ones((r, 8), device="cuda", dtype=t.bfloat16)
    w = t.zeros((8, c), device="cuda", dtype=t.bfloat16)
    w[0] = 1.0
    dx = t.empty_like(y)
    oba.linear_input_grad(dy, w, dx, oba.linear_workspace(r, c, 8), act=act, q=q, e=e)
    t.cuda.synchronize()
    close(dx, (p > 0).double(), 0.0, "act'")


# Bounds of the functions as they are evaluated, in units of 2^-24 of the
# value.  Phi(-z) = exp2(c z^2) P(t): the exponent's argument has three
# roundings and is 0.72 z^2 (1.5 z^2 of the value); the fit is 15 off, the
# hardware's exp2 and reciprocal 2 each, the polynomial and the products 10.
# (1 + tanh u) / 2 = 1 / (1 + exp2(a)): u and a have 8 roundings of an a that
# is 2 u log2(e), which matter as far as the exponential does.
UNIT = 2.0 ** -24


def phi_bound(p):
    return (32 + 1.5 * p * p) * UNIT


def sigmoid_bound(p):
    t = torch()
    u = math.sqrt(2 / math.pi) * (p + 0.044715 * p ** 3)
    return u, (8 + 16 * u.abs() * t.sigmoid(-2 * u)) * UNIT


@pytest.mark.parametrize("act,low", [("gelu", -13.0), ("gelu_tanh", -9.5)])
@pytest.mark.parametrize("r", [1, 130])
def test_accuracy_of_the_functions(r, act, low):
    """p is the bias alone, so it is any binary32 value; the residual is minus
    the rounded result, so what is stored is the function's own error and the
    rounding of a value 2^-8 as large."""
    t = torch()
    say(f"[act accuracy] {r} rows {act}")
    c = 8192
    p = t.linspace(low, 13.0, c, device="cuda")
    p6 = p.double()
    ref = act64(p6, act).expand(r, c)
    res = -ref.to(t.bfloat16).contiguous()
    x = t.zeros((r, 8), device="cuda", dtype=t.bfloat16)
    w = t.zeros((c, 8), device="cuda", dtype=t.bfloat16)
    y = t.empty((r, c), device="cuda", dtype=t.bfloat16)
    oba.linear(x, w, y, oba.linear_workspace(r, 8, c), bias=p, act=act, residual=res)
    t.cuda.synchronize()
    bound = (phi_bound(p6) if act == "gelu" else sigmoid_bound(p6)[1]) + 2 * UNIT
    diff = ref + res.double()
    err = bound * ref.abs()
    close(y, diff, err + half("bf16") * (diff.abs() + err) + 2.0 ** -126, "act")


@pytest.mark.parametrize("act,low", [("gelu", -13.0), ("gelu_tanh", -9.5)])
@pytest.mark.parametrize("r", [1, 130])
def test_accuracy_of_the_derivatives(r, act, low):
    t = torch()
    say(f"[act' accuracy] {r} rows {act}")
    c = 8192
    q, e = oba.act8_buffers(r, c)
    oba.act8_encode(t.linspace(low, 13.0, c, device="cuda").expand(r, c).contiguous(), q, e)
    t.cuda.synchronize()
    p = decode64(q, e, c)
    ref = act_grad64(p, act)
    res = -ref.to(t.bfloat16).contiguous()
    dy = t.ones((r, 8), device="cuda", dtype=t.bfloat16)
    w = t.zeros((8, c), device="cuda", dtype=t.bfloat16)
    w[0] = 1.0
    dx = t.empty_like(res)
    oba.linear_input_grad(dy, w, dx, oba.linear_workspace(r, c, 8), act=act, q=q, e=e, add=res)
    t.cuda.synchronize()
    if act == "gelu":
        cdf = 0.5 * t.erfc(-p / math.sqrt(2.0))
        err = phi_bound(p) * (cdf + (ref - cdf).abs()) + 2 * UNIT * ref.abs()
    else:
        u, es = sigmoid_bound(p)
        s = t.sigmoid(2 * u)
        d = math.sqrt(2 / math.pi) * (2 + 6 * 0.044715 * p * p)
        # 1 - s is off by s's error and a rounding; where the exponential is
        # below half a unit, s is 1 and 1 - s is 0
        e1 = t.where(t.exp(-2 * u) < 2.0 ** -25, t.sigmoid(-2 * u), s * es + UNIT)
        err = s * es + p.abs() * d * s * (t.sigmoid(-2 * u) * (es + 8 * UNIT) + e1) \
            + UNIT * ref.abs()
    diff = ref + res.double()
    close(dx, diff, err + half("bf16") * (diff.abs() + err) + 2.0 ** -126, "act'")
