"""The join between two blocks (norm, dropout, gate, residual sum, norm) and its
backward pass against plain binary64 forms: every type, both kinds of norm, every
part left out, widths of every number of waves, one row, no rows."""
import sys

import pytest

from communication_compressed_optimizer_02_amd import binding as oba
from layer_common import (check_kept, close, dt, encode64, gen, half, out_rows, rows, tiny, torch,
                          untouched)
from sublayer_common import (UNIT, factor_gpu, norm_rows64, norm_rows_bound, through64,
                             through_bound)

pytestmark = pytest.mark.gpu
TYPES = ("f32", "f16", "bf16")
COLS = [1, 7, 32, 500, 513, 1000, 1600, 2048, 2049, 4100, 8192, 8200, 16384]
ETA = 1e-5
SEED, STEP, SITE = 77, 5, 2
# post norm, pre norm, gate, betas, dropout's rate, alpha
FORMS = [(True, True, True, True, 0.1, 1.25), (False, True, False, False, 0.0, 1.0),
         (True, False, False, True, 0.3, 0.5), (False, True, True, True, 0.2, 1.0),
         (True, True, False, False, 0.0, -2.0), (False, False, True, False, 0.1, 1.0)]


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def vec(g, c, a, b):
    t = torch()
    return (a + b * t.randn(c + 1, generator=g, device="cuda"))[1:]  # at an odd place


def params(g, c, form):
    post, pre, gate, beta, _, _ = form
    return dict(gamma_b=vec(g, c, 1.0, 0.3) if post else None,
                beta_b=vec(g, c, 0.0, 0.3) if post and beta else None,
                gate=vec(g, c, 0.5, 0.3) if gate else None,
                gamma=vec(g, c, 1.0, 0.3) if pre else None,
                beta=vec(g, c, 0.0, 0.3) if pre and beta else None)


def forward(x, b, p, form, kind, r=True, keep=True):
    t = torch()
    post, pre, _, _, rate, alpha = form
    n, c = x.shape
    name = {v: k for k, v in {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}.items()}
    d = name[x.dtype]
    o = dict(r=out_rows(n, c, d) if r else (None, None),
             z=out_rows(n, c, d) if pre else (None, None),
             rstd=t.full((n,), 7.0, device="cuda") if pre else None,
             rstd_b=t.full((n,), 7.0, device="cuda") if post else None,
             kept=oba.act8_buffers(n, c) if keep and pre else (None, None),
             kept_b=oba.act8_buffers(n, c) if keep and b is not None else (None, None))
    oba.residual_norm(x, ETA, b=b, alpha=alpha, gate=p["gate"], gamma_b=p["gamma_b"],
                      beta_b=p["beta_b"], rstd_b=o["rstd_b"], qb=o["kept_b"][0],
                      eb=o["kept_b"][1], rate=rate, rng=oba.dropout_rng(SEED, STEP), site=SITE,
                      r=o["r"][0], gamma=p["gamma"], beta=p["beta"], z=o["z"][0], rstd=o["rstd"],
                      q=o["kept"][0], e=o["kept"][1], kind=kind)
    t.cuda.synchronize()
    return o


def check_forward(x, b, p, form, kind, o, dtype):
    post, pre, gate, beta, rate, alpha = form
    n, c = x.shape
    h = half(dtype) * (1 + 2 ** -7)
    one = lambda v, d: d if v is None else v.double()  # noqa: E731
    x6 = x.double()
    v, ev = b.double(), torch().zeros_like(x6)
    if post:
        rs = norm_rows64(v, ETA, kind)[1]
        ev, rel = norm_rows_bound(v, ev, ETA, kind)
        v = norm_rows64(v, ETA, kind)[0]
        close(o["rstd_b"], rs[:, 0], (rs * (rel + UNIT))[:, 0], "rstd_b")
    if o["kept_b"][0] is not None:
        check_kept(*o["kept_b"], v, ev, "branch")
    if post:
        g, s = p["gamma_b"].double(), one(p["beta_b"], 0.0)
        v, ev = v * g + s, ev * g.abs()
        ev = ev + UNIT * v.abs()
    f = factor_gpu(n, c, rate, SEED, STEP, SITE)
    v, ev = v * f, ev * f + 2 * UNIT * (v * f).abs()
    if gate:
        v, ev = v * p["gate"].double(), ev * p["gate"].double().abs()
        ev = ev + UNIT * v.abs()
    r = alpha * x6 + v
    er = ev + UNIT * ((alpha * x6).abs() + r.abs())
    if o["r"][0] is not None:
        close(o["r"][0], r, er + h * r.abs() + tiny(dtype), "r")
        untouched(o["r"][1], c)
    if pre:
        k, rs = norm_rows64(r, ETA, kind)
        ek, rel = norm_rows_bound(r, er, ETA, kind)
        close(o["rstd"], rs[:, 0], (rs * (rel + UNIT) * (1 + rel))[:, 0], "rstd")
        if o["kept"][0] is not None:
            check_kept(*o["kept"], k, ek, "normalised rows")
        g, s = p["gamma"].double(), one(p["beta"], 0.0)
        z = k * g + s
        close(o["z"][0], z, ek * g.abs() + UNIT * z.abs() + h * z.abs() + tiny(dtype), "z")
        untouched(o["z"][1], c)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("c", COLS)
def test_forward_widths(c, dtype):
    t = torch()
    n = 37 if c < 4000 else 5
    kind = "layer" if (c + len(dtype)) % 2 else "rms"
    say(f"[join] {n}x{c} {dtype} {kind}")
    g = gen(c)
    x, b = rows(g, n, c, dtype, extra=8), rows(g, n, c, dtype, std=0.5)
    b += (3.0 * t.randn((n, 1), generator=g, device="cuda")).to(b.dtype)
    p = params(g, c, FORMS[0])
    o = forward(x, b, p, FORMS[0], kind)
    check_forward(x, b, p, FORMS[0], kind, o, dtype)
    # nothing kept: the same values
    o2 = forward(x, b, p, FORMS[0], kind, keep=False)
    assert t.equal(o["r"][0], o2["r"][0]) and t.equal(o["z"][0], o2["z"][0])
    assert t.equal(o["rstd"], o2["rstd"]) and t.equal(o["rstd_b"], o2["rstd_b"])


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,c,dtype", [(1, 1600, "bf16"), (67, 200, "f16"), (1030, 96, "f32"),
                                       (9, 5000, "bf16")])
def test_forward_forms(n, c, dtype, form, kind):
    say(f"[join] {n}x{c} {dtype} {kind} {form}")
    g = gen(n + c)
    x, b = rows(g, n, c, dtype, extra=8), rows(g, n, c, dtype, std=0.5)
    p = params(g, c, form)
    o = forward(x, b, p, form, kind)
    check_forward(x, b, p, form, kind, o, dtype)
    if form[1]:  # r itself not wanted
        o2 = forward(x, b, p, form, kind, r=False)
        assert torch().equal(o["z"][0], o2["z"][0])


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("c", [40, 700, 3000, 9000])
def test_a_norm_alone(c, kind):
    """Without a branch: r = alpha x and its norm."""
    t = torch()
    g = gen(c)
    x = rows(g, 11, c, "bf16")
    gamma = vec(g, c, 1.0, 0.3)
    z, buf = out_rows(11, c, "bf16")
    r, _ = out_rows(11, c, "bf16")
    rstd = t.empty(11, device="cuda")
    oba.residual_norm(x, ETA, alpha=2.0, r=r, gamma=gamma, z=z, rstd=rstd, kind=kind)
    t.cuda.synchronize()
    r6 = 2.0 * x.double()
    assert t.equal(r, r6.bfloat16())
    h, rs = norm_rows64(r6, ETA, kind)
    eh, rel = norm_rows_bound(r6, t.zeros_like(r6), ETA, kind)
    close(rstd, rs[:, 0], (rs * (rel + UNIT))[:, 0], "rstd")
    ref = h * gamma.double()
    close(z, ref, eh * gamma.double().abs() + (UNIT + half("bf16") * (1 + 2 ** -7)) * ref.abs()
          + tiny("bf16"), "z")
    untouched(buf, c)


@pytest.mark.parametrize("c", [64, 777, 1500, 6000, 12000])
def test_rows_far_from_zero_and_constant_rows(c):
    """The mean of 10^4 spreads, and rows of one value: their centred values are 0."""
    t = torch()
    g = gen(c)
    x, b = (t.zeros((6, (c + 7) // 8 * 8), device="cuda")[:, :c] for _ in range(2))
    b += t.randn((6, c), generator=g, device="cuda") * 0.25 + 2500.0
    b[3], b[4] = 1234.567, -3e-5
    form = (True, False, False, False, 0.0, 0.0)
    p = params(g, c, form)
    o = forward(x, b, p, form, "layer")
    check_forward(x, b, p, form, "layer", o, "f32")
    assert bool((o["r"][0][3:5] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("c", [500, 777, 1600, 5000, 9001])
def test_large_constant_rows_stay_finite(c, dtype):
    """A row of one large value of 24 bits: its squares around the mean are a difference of equal
    sums and may not become less than 0.  Its centred values are what the mean is off
    by, at most 20 units of the first sum's error of 20 units, over sqrt(eta)."""
    t = torch()
    vals = 10 ** (t.rand(300, generator=gen(c), device="cuda") * (2 if dtype == "f16" else 13) + 2)
    buf = t.zeros((300, (c + 7) // 8 * 8), device="cuda", dtype=dt(dtype))
    buf[:, :c] = vals[:, None].to(dt(dtype))
    z, rstd = t.empty_like(buf)[:, :c], t.zeros(300, device="cuda")
    oba.residual_norm(buf[:, :c], ETA, alpha=1.1, gamma=t.ones(c, device="cuda"), z=z, rstd=rstd)
    t.cuda.synchronize()
    assert bool(t.isfinite(z).all()) and bool((rstd > 0).all())
    off = 0 if dtype == "f32" else 440 * UNIT * UNIT * buf[:, :1].double() / ETA ** 0.5
    assert bool((z.double().abs() <= off * (1 + 2 ** -7)).all())


def test_infinities_and_nan_stay_in_their_rows():
    t = torch()
    for kind in ("layer", "rms"):
        for c in (300, 1700):
            g = gen(c)
            x, b = rows(g, 40, c, "bf16"), rows(g, 40, c, "bf16")
            p = params(g, c, FORMS[4])
            clean = forward(x, b, p, FORMS[4], kind)
            b[7, 5], b[8, c - 1], x[9, 0] = float("inf"), float("nan"), float("-inf")
            o = forward(x, b, p, FORMS[4], kind)
            bad = t.zeros(40, dtype=t.bool, device="cuda")
            bad[7:10] = True
            for name in ("r", "z"):
                assert t.equal(o[name][0][~bad], clean[name][0][~bad])
                assert bool((~t.isfinite(o[name][0][bad])).any(1).all()), name
            assert bool((o["kept"][1][bad] == 255).any(1).all())


# ---- backward -----------------------------------------------------------------------------

def backward(n, c, per, dtype, form, kind, gt, with_dr=True, want=True, db=True):
    """Inputs, the call and everything it gave."""
    t = torch()
    post, pre, gate, beta, rate, alpha = form
    total = n * per
    g = gen(n + c * 3 + per)
    p = params(g, c, form)
    s = dict(p=p)
    if pre:
        s["dz"] = rows(g, total, c, dtype, std=0.25, extra=8)
        s["q"], s["e"], s["h"] = encode64(rows(g, total, c, "f32"))
        s["rstd"] = t.rand(total, generator=g, device="cuda") + 0.5
    s["dr"] = rows(g, total, c, dtype, std=0.25) if with_dr or not pre else None
    s["qb"], s["eb"], s["k"] = encode64(rows(g, total, c, "f32"))
    if post:
        s["rstd_b"] = t.rand(total, generator=g, device="cuda") + 0.5
    names = [k for k, on in (("gamma", pre), ("beta", pre), ("gate", gate), ("gamma_b", post),
                             ("beta_b", post)) if on] if want else []
    at = {k: 3 + i * (c + 1) for i, k in enumerate(names)}
    ld = (3 + 5 * (c + 1) + 15) // 8 * 8
    s["grads"] = t.full((n, ld), 7.0, device="cuda", dtype=dt(gt))
    s["at"] = at
    s["dx"], s["dxbuf"] = out_rows(total, c, dtype)
    s["db"], s["dbbuf"] = out_rows(total, c, dtype) if db else (None, None)
    ws = oba.residual_norm_backward_workspace(n, per, c)
    oba.residual_norm_backward(
        n, s["dx"], s["grads"], ws if want else None, dz=s.get("dz"), dr=s["dr"], alpha=alpha,
        q=s.get("q"), e=s.get("e"), rstd=s.get("rstd"), gamma=p["gamma"], at_gamma=at.get("gamma"),
        at_beta=at.get("beta"), db=s["db"], qb=s["qb"], eb=s["eb"], rstd_b=s.get("rstd_b"),
        gamma_b=p["gamma_b"], beta_b=p["beta_b"], gate=p["gate"], at_gate=at.get("gate"),
        at_gamma_b=at.get("gamma_b"), at_beta_b=at.get("beta_b"), rate=rate,
        rng=oba.dropout_rng(SEED, STEP), site=SITE, kind=kind)
    t.cuda.synchronize()
    return s


def check_backward(s, n, c, per, dtype, form, kind, gt):
    t = torch()
    post, pre, gate, beta, rate, alpha = form
    p, total = s["p"], n * per
    h = half(dtype) * (1 + 2 ** -7)
    zero = t.zeros((total, c), dtype=t.float64, device="cuda")
    d, ed = zero, zero
    sums = {}
    if pre:
        dz, a = s["dz"].double(), s["dz"].double() * p["gamma"].double()
        sums["gamma"], sums["beta"] = (dz * s["h"], zero), (dz, zero)
        rs = s["rstd"].double()[:, None]
        d = through64(a, s["h"], rs, kind)
        ed = through_bound(a, UNIT * a.abs(), s["h"], rs, kind)
    if s["dr"] is not None:
        d = d + s["dr"].double()
        ed = ed + UNIT * (d.abs() + (d - s["dr"].double()).abs())
    ref = alpha * d
    close(s["dx"], ref, abs(alpha) * ed + (2 * UNIT + h) * ref.abs() + tiny(dtype), "dx")
    untouched(s["dxbuf"], c)
    f = factor_gpu(total, c, rate, SEED, STEP, SITE)
    v, ev = d * f, ed * f + 2 * UNIT * (d * f).abs()
    gb = p["gamma_b"].double() if post else 1.0
    gt_ = p["gate"].double() if gate else 1.0
    sums["S"], sums["T"] = (v * s["k"], ev * s["k"].abs()), (v, ev)
    if s["db"] is not None:
        w, ew = v * gt_ * gb, ev * abs(gt_ * gb) if gate or post else ev
        ew = ew + 2 * UNIT * w.abs()
        if post:
            rs = s["rstd_b"].double()[:, None]
            w, ew = through64(w, s["k"], rs, kind), through_bound(w, ew, s["k"], rs, kind)
        close(s["db"], w, ew + (UNIT + h) * w.abs() + tiny(dtype), "db")
        untouched(s["dbbuf"], c)

    def total_of(name):
        term, err = sums[name]
        term, err = term.reshape(n, per, c), err.reshape(n, per, c)
        # a binary32 sum of at most `per` terms, then binary64
        return term.sum(1), err.sum(1) + (per + 2) * UNIT * term.abs().sum(1)

    hg = half(gt) * (1 + 2 ** -7)
    bb = p["beta_b"].double() if p["beta_b"] is not None else 0.0
    seen = t.zeros_like(s["grads"], dtype=t.bool)
    for name, at in s["at"].items():
        if name in ("gamma", "beta"):
            want, err = total_of(name)
        else:
            (S, eS), (T, eT) = total_of("S"), total_of("T")
            if name == "gate":
                want, err = S * gb + T * bb, eS * abs(gb) + eT * abs(bb)
            else:
                want, err = (S * gt_, eS * abs(gt_)) if name == "gamma_b" else \
                    (T * gt_, eT * abs(gt_))
        got = s["grads"][:, at:at + c]
        seen[:, at:at + c] = True
        close(got, want, err + (hg + UNIT) * want.abs() + tiny(gt), "d" + name)
    assert bool((s["grads"][~seen] == 7.0).all()), "other gradients of the rows were written"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("c", COLS)
def test_backward_widths(c, dtype):
    per = 19 if c < 4000 else 3
    kind = "layer" if (c + len(dtype)) % 2 else "rms"
    gt = TYPES[c % 3]
    say(f"[join backward] 2x{per}x{c} {dtype} {kind} -> {gt}")
    s = backward(2, c, per, dtype, FORMS[0], kind, gt)
    check_backward(s, 2, c, per, dtype, FORMS[0], kind, gt)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,per,c,dtype,gt", [(1, 1, 1600, "bf16", "f32"),
                                              (3, 101, 200, "f16", "f16"),
                                              (5, 1300, 40, "f32", "f32"),
                                              (7, 2, 2100, "bf16", "bf16")])
def test_backward_forms(n, per, c, dtype, gt, form, kind):
    say(f"[join backward] {n}x{per}x{c} {dtype} -> {gt} {kind} {form}")
    s = backward(n, c, per, dtype, form, kind, gt)
    check_backward(s, n, c, per, dtype, form, kind, gt)
    if form[1]:
        s = backward(n, c, per, dtype, form, kind, gt, with_dr=False)
        check_backward(s, n, c, per, dtype, form, kind, gt)
    # the parameters' gradients, or the branch's, not wanted: the others the same
    a = backward(n, c, per, dtype, form, kind, gt, want=False)
    b = backward(n, c, per, dtype, form, kind, gt)
    d = backward(n, c, per, dtype, form, kind, gt, db=False)
    assert torch().equal(a["dx"], b["dx"]) and torch().equal(a["db"], b["db"])
    assert torch().equal(d["dx"], b["dx"]) and torch().equal(d["grads"], b["grads"])
    assert bool((a["grads"] == 7.0).all())


def test_no_rows():
    t = torch()
    x = t.empty((0, 40), device="cuda")
    v, p = t.empty(0, device="cuda"), t.ones(40, device="cuda")
    q, e = oba.act8_buffers(0, 40)
    oba.residual_norm(x, ETA, b=x, r=x, gamma=p, z=x, rstd=v, q=q, e=e)
    grads = t.full((2, 208), 7.0, device="cuda")
    oba.residual_norm_backward(2, x, grads, None, dz=x, q=q, e=e, rstd=v, gamma=p, at_gamma=0,
                               at_beta=40, qb=q, eb=e, rstd_b=v, gamma_b=p, at_gamma_b=80,
                               at_beta_b=120, gate=p, at_gate=160)
    t.cuda.synchronize()
    assert bool((grads[:, :200] == 0).all()) and bool((grads[:, 200:] == 7.0).all())


def test_gradients_against_differences():
    """Forward passes in binary64 at both sides of the inputs and parameters, the
    same mask: a product's slope along random directions."""
    t = torch()
    n, c, form = 6, 77, FORMS[0]
    for kind in ("layer", "rms"):
        g = gen(3)
        x, b = rows(g, n, c, "f32", pad=0.0), rows(g, n, c, "f32", pad=0.0)
        p = params(g, c, form)
        dz, dr = rows(g, n, c, "f32", pad=0.0), rows(g, n, c, "f32", pad=0.0)
        f = factor_gpu(n, c, form[4], SEED, STEP, SITE)
        names = ("gamma_b", "beta_b", "gate", "gamma", "beta")
        args = [x.double(), b.double()] + [p[k].double() for k in names]
        dirs = [t.randn(v.shape, generator=g, device="cuda").double() for v in args]

        def value(h):
            xv, bv, gb, bb, ga, gm, be = (v + h * d for v, d in zip(args, dirs))
            r = form[5] * xv + ga * (f * (norm_rows64(bv, ETA, kind)[0] * gb + bb))
            z = norm_rows64(r, ETA, kind)[0] * gm + be
            return float((z * dz.double()).sum() + (r * dr.double()).sum())

        h = 1e-6
        slope = (value(h) - value(-h)) / (2 * h)
        # the backward pass from rows kept in 8 bits: exact for rows that are
        # integers of a group's step, so the kept rows are what is differentiated
        k, rsb = norm_rows64(args[1], ETA, kind)
        v = f * (k * args[2] + args[3])
        r = form[5] * args[0] + args[4] * v
        hh, rs = norm_rows64(r, ETA, kind)
        d = through64(dz.double() * args[5], hh, rs, kind) + dr.double()
        e = d * f
        exact = [form[5] * d, through64(e * args[4] * args[2], k, rsb, kind),
                 (e * args[4] * k).sum(0), (e * args[4]).sum(0),
                 (e * (k * args[2] + args[3])).sum(0), (dz.double() * hh).sum(0),
                 dz.double().sum(0)]
        scale = sum(float((a * w).abs().sum()) for a, w in zip(exact, dirs))
        formula = sum(float((a * w).sum()) for a, w in zip(exact, dirs))
        assert abs(slope - formula) <= 1e-7 * scale
        # and the call's gradients are near the formula's: what 8 bits change is at
        # most 2^-7 of a group's largest value, in h and in k
        o = forward(x, b, p, form, kind)
        grads = t.zeros((1, 5 * c + 3), device="cuda")
        dx, db = out_rows(n, c, "f32")[0], out_rows(n, c, "f32")[0]
        oba.residual_norm_backward(
            1, dx, grads, oba.residual_norm_backward_workspace(1, n, c), dz=dz, dr=dr,
            alpha=form[5], q=o["kept"][0], e=o["kept"][1], rstd=o["rstd"], gamma=p["gamma"],
            at_gamma=3 * c, at_beta=4 * c, db=db, qb=o["kept_b"][0], eb=o["kept_b"][1],
            rstd_b=o["rstd_b"], gamma_b=p["gamma_b"], beta_b=p["beta_b"], gate=p["gate"],
            at_gate=2 * c, at_gamma_b=0, at_beta_b=c, rate=form[4],
            rng=oba.dropout_rng(SEED, STEP), site=SITE, kind=kind)
        t.cuda.synchronize()
        got = [dx, db] + [grads[0, i * c:(i + 1) * c] for i in range(5)]
        for a, w, what in zip(got, exact, ("dx", "db", *names)):
            rel = float((a.double() - w).norm() / w.norm())
            assert rel <= 4 * 2.0 ** -6, f"{what}: {rel}"
