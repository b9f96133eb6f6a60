"""The activation functions and their derivatives over all of binary32's
range."""
import sys

import pytest

from communication_compressed_optimizer_02_amd import binding as oba
from layer_common import close, decode64, half, torch

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
