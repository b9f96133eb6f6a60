"""The stack's gradients against differences of its binary64 model, a tensor and a
worker at a time."""
import pytest

import test_gpu_gated_feedforward as gff
from layer_common import torch
from sublayer_common import factor_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", gff.FORMS)
def test_slopes_along_the_gradient(form):
    """Along the model's own gradient the slope is that gradient's norm, and the
    kernels', off by 0.3 of it in norm at most (test_a_pass_against_the_model
    derives it), has a slope that is off by 0.3 of it at most.  Of a direction that a
    gradient has nothing to do with the slope is 0.  A central difference of a step of
    1e-5 of the tensor's norm is off by 1e-10 of the third derivative, and by what
    rounds in binary64, 1e-16 / 1e-5."""
    t = torch()
    n, r, width = 2, 65, 64
    gff.say(f"[gff] slopes {form}")
    F, L, S, x, dy = gff.make(width, 160, n, r, 40 + len(form), **form)
    F.forward(x)
    dx = F.backward(dy, S.g)
    t.cuda.synchronize()
    seed, step = (int(v) for v in F.rng.cpu())
    masks = [factor_gpu(n * r, width, F.rate, seed, step, F.site + k) for k in range(F.layers)]
    p = gff.params64(F, S.x)
    for i in range(n):
        part = slice(i * r, (i + 1) * r)

        def loss(xx):
            out = gff.model64(F, xx, p, [m[part] for m in masks])
            return (out * dy.double()[part]).sum()

        tensors = {(k, name): v for k, q in enumerate(p) for name, v in q.items()}
        got = {(k, name): F.part(S.g[i], k, name).double().view(v.shape)
               for (k, name), v in tensors.items()}
        xx = x.double()[part].clone()
        tensors["x"], got["x"] = xx, dx.double()[part]
        for v in tensors.values():
            v.grad = None
            v.requires_grad_(True)
        loss(xx).backward()
        for v in tensors.values():
            v.requires_grad_(False)
        for key, v in tensors.items():
            along = v.grad / v.grad.norm()
            h = 1e-5 * float(v.norm().clamp(min=1.0))
            at = v.clone()
            f = []
            for s in (h, -h):
                v.copy_(at + s * along)
                f.append(float(loss(xx)))
            v.copy_(at)
            diff = (f[0] - f[1]) / (2 * h)
            slope = float((got[key] * along).sum())
            assert diff > 0 and abs(diff - slope) <= 0.3 * diff, (i, key, diff, slope)
    L.close()
