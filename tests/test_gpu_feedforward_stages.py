"""The feed-forward sub-layer's first stage and kept tensors against binary64,
and the whole pass, without an activation, against the binary64 function's own
gradients.  (With one, the derivative at a pre-activation of 8 bits moves the
gradients by more than a worst-case bound through the norm tells apart; there
each stage is held against its formula.)"""
import sys

import pytest

from communication_compressed_optimizer_02_amd import FeedForward, synth
from communication_compressed_optimizer_02_amd import binding as oba
from layer_common import (GROUP, U, check_kept, close, encode64, gen, half, norm64, norm_grad64,
                          rows, tiny, torch)

pytestmark = pytest.mark.gpu
CASES = [(64, 256, 2, 33, "bf16", "gelu"), (100, 300, 3, 70, "f16", "gelu_tanh"),
         (40, 72, 1, 1, "bf16", "relu"), (136, 264, 4, 129, "f16", "none")]
ETA = 0.05  # beside rows of variance 0.1: a norm with another eta is another norm


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def make(width, hidden, n, r, dtype, act, seed, gt="f32", std=0.3):
    F = FeedForward(width, hidden, n, r, dtype, act, eta=ETA)
    L = oba.Layout(F.size, n, synth.whole(F.size), synth.even_shards(F.size, n))
    S = oba.State(L, gt)
    g = gen(seed)
    F.init(S.x, g)
    F.part(S.x, "gamma").normal_(1.0, 0.2, generator=g)
    for name in ("beta", "b1", "b2"):
        F.part(S.x, name).normal_(0.0, 0.3, generator=g)
    F.load(S.x)
    return F, L, S, rows(g, n * r, width, dtype, std=std), rows(g, n * r, width, dtype, std=0.1)


def norm_bounds(x):
    """mean, rstd, xhat and their errors: 50 additions a sum, as the norm's own
    tests have them, of values that are of the spread's size."""
    m, s, z = norm64(x, ETA)
    big = x.double().abs().amax(1)
    es = s * 80 * U * (1 + big * s)
    h = z * s[:, None]
    eh = 60 * U * big[:, None] * s[:, None] + h.abs() * (es / s)[:, None] + 3 * U * h.abs()
    return m, s, h, 52 * U * big, es, eh


@pytest.mark.parametrize("width,hidden,n,r,dtype,act", CASES)
def test_norm_and_kept_tensors(width, hidden, n, r, dtype, act):
    t = torch()
    say(f"[ff stages] {width}x{hidden} n={n} rows={r} {dtype} {act}")
    F, L, S, x, dy = make(width, hidden, n, r, dtype, act, width + r)
    F.forward(x)
    t.cuda.synchronize()
    p = {k: F.part(S.x, k).double() for k in F.places}
    m, s, h, em, es, eh = norm_bounds(x)
    close(F.rstd, s, es, "rstd")
    check_kept(*F.kept_norm, h, eh, "xhat")
    hb = half(dtype) * (1 + 2 ** -7)

    def z_of(gamma, beta, hat, ehat):
        ref = hat * gamma + beta
        return ref, ehat * gamma.abs() + 4 * U * ((hat * gamma).abs() + ref.abs()) \
            + hb * ref.abs() + tiny(dtype)

    ref, err = z_of(p["gamma"], p["beta"], h, eh)
    close(F.z, ref, err, "z")
    # the bound tells the parameters apart, and eta from the default
    other, _ = z_of(p["beta"], p["gamma"], h, eh)
    assert bool(((F.z.double() - other).abs() > err).any())
    assert bool(((s - norm64(x, 1e-5)[1]).abs() > es).all())
    q, e, _ = encode64(F.z)
    assert t.equal(q, F.kept_z[0]) and t.equal(e, F.kept_z[1]), "the first product's input"
    if act != "none":
        z, w1 = F.z.double(), F.w1.double()
        pre = z @ w1.t() + p["b1"]
        ep = (width + 2) * U * (z.abs() @ w1.abs().t()) + U * (pre.abs() + p["b1"].abs()) + 1e-30
        check_kept(*F.kept_pre, pre, ep, "pre-activation")
    assert t.equal(F.w1.float(), F.part(S.x, "w1").view(hidden, width).to(F.dtype).float())
    assert t.equal(F.w2.float(), F.part(S.x, "w2").view(width, hidden).to(F.dtype).float())
    L.close()


def per_worker(n, a, b):
    """Every worker's a^T b."""
    return torch().bmm(a.reshape(n, -1, a.shape[1]).transpose(1, 2).contiguous(),
                       b.reshape(n, -1, b.shape[1]).contiguous())


def sums(n, a):
    return a.reshape(n, -1, a.shape[1]).sum(1)


def whole(n, x, u, q):
    """The binary64 function at these parameters: sum(u * y), its intermediate
    results and its gradients (those of the parameters per worker)."""
    _, s, z = norm64(x, ETA)
    v = dict(s=s, h=z * s[:, None])
    v["z"] = v["h"] * q["gamma"] + q["beta"]
    v["p"] = v["z"] @ q["w1"].t() + q["b1"]
    v["f"] = float((u * (v["p"] @ q["w2"].t() + q["b2"] + x)).sum())
    v["dh"] = u @ q["w2"]
    v["dz"] = v["dh"] @ q["w1"]
    dx, dg, db = norm_grad64(n, v["dz"], q["gamma"], s, v["h"], u)
    return v, dict(x=dx, gamma=dg, beta=db, w1=per_worker(n, v["dh"], v["z"]),
                   b1=sums(n, v["dh"]), w2=per_worker(n, u, v["p"]), b2=sums(n, u))


def bounds(n, r, x, u, q, dtype, v, ref):
    """What each gradient may be off by: each rounding to 16 bits (half a step)
    and to 8 (a step, at most 1/64 of its group's largest magnitude) carried
    through the formulas."""
    t = torch()
    hidden, width = q["w1"].shape
    hb = half(dtype) * (1 + 2 ** -7)

    def in8(a, e):
        """the error of a, of error e, once it is kept in 8 bits"""
        c = a.shape[1]
        p = t.zeros((a.shape[0], -(-c // GROUP) * GROUP), dtype=t.float64, device=x.device)
        p[:, :c] = a.abs() + e
        top = p.view(p.shape[0], -1, GROUP).amax(2) / 64 + 2.0 ** -126
        return e + top.repeat_interleave(GROUP, dim=1)[:, :c]

    w1, w2, gamma, ua = q["w1"].abs(), q["w2"].abs(), q["gamma"].abs(), u.abs()
    _, s, h, _, es, eh = norm_bounds(x)
    za, pa, ha, da, qa = (v[k].abs() for k in ("z", "p", "h", "dh", "dz"))
    ez = eh * gamma + (hb + 8 * U) * (za + gamma * ha + 1e-6)
    ep = ez @ w1.t() + (width + 4) * U * ((za + ez) @ w1.t() + q["b1"].abs())
    ep = ep + hb * (pa + ep) + tiny(dtype)
    z8, p8, h8 = in8(v["z"], ez), in8(v["p"], ep), in8(h, eh)
    ed = (width + 2) * U * (ua @ w2)
    ed = ed + hb * (da + ed) + tiny(dtype)
    eq = ed @ w1 + (hidden + 2) * U * ((da + ed) @ w1)
    eq = eq + hb * (qa + eq) + tiny(dtype)
    k = (r + 8) * U  # the additions of a gradient's sums
    err = dict(w2=per_worker(n, ua, p8 + k * (pa + p8)), b2=k * sums(n, ua),
               w1=per_worker(n, ed + k * (da + ed), za + z8) + per_worker(n, da, z8),
               b1=sums(n, ed + k * (da + ed)),
               gamma=sums(n, eq * (ha + h8) + qa * h8 + k * (qa + eq) * (ha + h8)),
               beta=sums(n, eq + k * (qa + eq)))
    a, ea = qa * gamma, eq * gamma + U * qa * gamma
    m1, m2 = a.mean(1, keepdim=True), (a * ha).mean(1, keepdim=True)
    em2 = (ea * (ha + h8) + a * h8).mean(1, keepdim=True)
    ex = s[:, None] * (ea + ea.mean(1, keepdim=True) + h8 * (m2 + em2) + ha * em2
                       + 120 * U * (a + m1 + ha * m2))
    ex = ex + (es / s)[:, None] * (ref["x"] - u).abs() * 2 + 2 * U * ua
    err["x"] = ex + hb * (ref["x"].abs() + ex) + tiny(dtype)
    return err


def planted(n, x, u, q, v, right):
    """The gradients of wrong passes, made from the formulas."""
    a = (v["dz"] * q["gamma"]).mean(1, keepdim=True)
    return {"gamma and beta swapped":
            whole(n, x, u, {**q, "gamma": q["beta"], "beta": q["gamma"]})[1],
            "no mean of the gradient": {**right, "x": right["x"] + v["s"][:, None] * a},
            "workers swapped": {k: g if k == "x" else g.flip(0) for k, g in right.items()},
            "no residual": {**right, "x": right["x"] - u},
            "no b1": whole(n, x, u, {**q, "b1": 0 * q["b1"]})[1]}


@pytest.mark.parametrize("width,hidden,n,r,dtype", [(136, 264, 4, 129, "f16"),
                                                    (72, 40, 2, 50, "bf16")])
def test_whole_pass_against_the_function(width, hidden, n, r, dtype):
    """dx and all six gradients against those of the binary64 function of x and
    the parameters, which are checked against its differences first."""
    t = torch()
    say(f"[ff whole] {width}x{hidden} n={n} rows={r} {dtype}")
    F, L, S, x, dy = make(width, hidden, n, r, dtype, "none", width + 2 * r)
    F.forward(x)
    dx = F.backward(dy, S.g)
    t.cuda.synchronize()
    q = {k: F.part(S.x, k).double() for k in ("gamma", "beta", "b1", "b2")}
    q["w1"], q["w2"] = F.w1.double(), F.w2.double()
    x6, u = x.double(), dy.double()
    v, ref = whole(n, x6, u, q)
    g = gen(9)
    d = {k: t.randn(a.shape, generator=g, device="cuda").double() for k, a in q.items()}
    dX, step = t.randn(x6.shape, generator=g, device="cuda").double(), 1e-6
    up, dn = (whole(n, x6 + k * dX, u, {i: q[i] + k * d[i] for i in q})[0]["f"]
              for k in (step, -step))
    terms = [ref["x"] * dX] + [ref[k].sum(0) * d[k] for k in q]
    # step^2 of the third derivative and 1e-16 / step of the sum's terms
    size = sum(float(a.abs().sum()) for a in terms) + float(u.abs().sum() * v["p"].abs().amax())
    assert abs((up - dn) / (2 * step) - sum(float(a.sum()) for a in terms)) <= 1e-6 * size
    err = bounds(n, r, x, u, q, dtype, v, ref)
    got = {name: F.part(S.g.t(), name).t() for name in err if name != "x"}
    got["x"] = dx
    for name, e in err.items():
        b = ref[name].reshape(-1, ref[name].shape[-1])
        close(got[name].reshape(b.shape), b, e.reshape(b.shape) + U * b.abs() + 1e-12, name)
    # the bound tells mistakes apart: each moves some gradient past twice of it
    for name, bad in planted(n, x6, u, q, v, ref).items():
        assert any(bool(((bad[k] - ref[k]).abs() > 2 * err[k].reshape(ref[k].shape)).any())
                   for k in ref), f"{name} would pass"
    L.close()
