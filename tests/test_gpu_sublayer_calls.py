"""How the gated sub-layer's operators may be called: matrices past 2^31 elements,
every number of waves to a row, strided slices, other streams, two at once,
captured and replayed, graphs that share a workspace, the smallest sizes."""
import sys

import pytest

from communication_compressed_optimizer_02_amd import binding as oba
from layer_common import U, close, dt, encode64, gen, half, out_rows, rows, tiny, torch
from sublayer_common import UNIT, gate64, gate_bounds

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def vec(g, c, about=0.0):
    return torch().randn(c, generator=g, device="cuda") * 0.2 + about


class Calls:
    """All five operators on the sizes of one sub-layer, with results of their own."""

    def __init__(self, seed, r=96, width=200, hidden=328, dtype="bf16", n=2, ws=None, **cut):
        t = torch()
        g = gen(seed)
        self.n, self.rng = n, oba.dropout_rng(seed, 3)
        self.x, self.b = rows(g, r, width, dtype, **cut), rows(g, r, width, dtype, **cut)
        self.w, self.w2 = (rows(g, 2 * hidden, width, dtype, std=width ** -0.5, **cut),
                           rows(g, width, hidden, dtype, std=hidden ** -0.5, **cut))
        self.par = {k: vec(g, width, k in ("gamma", "gamma_b", "gate"))
                    for k in ("gamma", "beta", "gamma_b", "beta_b", "gate")}
        self.bias = vec(g, 2 * hidden)
        new = lambda c: out_rows(r, c, dtype)[0]  # noqa: E731
        self.y, self.r, self.z, self.h = new(width), new(width), new(width), new(hidden)
        self.dpu, self.dx, self.db = new(2 * hidden), new(width), new(width)
        self.rs = [t.zeros(r, device="cuda") for _ in range(2)]
        self.kept = [oba.act8_buffers(r, width) for _ in range(2)]
        self.pu = [oba.act8_buffers(r, hidden) for _ in range(3)]
        self.g = t.zeros((n, 5 * width), device="cuda", dtype=dt("f16"))
        self.ws = ws if ws is not None else max(
            (oba.gated_linear_workspace(r, width, hidden),
             oba.gated_hidden_grad_workspace(r, hidden, width),
             oba.residual_norm_backward_workspace(n, r // n, width)), key=lambda v: v.numel())

    def run(self, **k):
        w = self.x.shape[1]
        oba.dropout(self.x, self.y, self.rng, 0.3, site=1, add=self.b, **k)
        (q, e), (qb, eb) = self.kept
        oba.residual_norm(self.x, 1e-5, b=self.b, alpha=0.5, rate=0.2, rng=self.rng, site=2,
                          rstd_b=self.rs[1], qb=qb, eb=eb, r=self.r, z=self.z, rstd=self.rs[0],
                          q=q, e=e, **self.par, **k)
        (qp, ep), (qu, eu), (qh, eh) = self.pu
        oba.gated_linear(self.z, self.w, self.h, self.ws, bias=self.bias, qp=qp, ep=ep, qu=qu,
                         eu=eu, q=qh, e=eh, **k)
        oba.gated_hidden_grad(self.b, self.w2, qp, ep, qu, eu, self.dpu, self.ws, **k)
        p = self.par
        oba.residual_norm_backward(
            self.n, self.dx, self.g, self.ws, dz=self.z, dr=self.x, alpha=0.5, q=q, e=e,
            rstd=self.rs[0], gamma=p["gamma"], at_gamma=0, at_beta=w, db=self.db, qb=qb, eb=eb,
            rstd_b=self.rs[1], gamma_b=p["gamma_b"], beta_b=p["beta_b"], gate=p["gate"],
            at_gate=2 * w, at_gamma_b=3 * w, at_beta_b=4 * w, rate=0.2, rng=self.rng, site=2, **k)

    def results(self):
        out = [self.y, self.r, self.z, self.h, self.dpu, self.dx, self.db, self.g, *self.rs]
        return out + [v for pair in self.kept + self.pu for v in pair]

    def copy(self):
        return [v.clone() for v in self.results()]

    def wipe(self):
        for v in self.results():
            v.zero_()

    def same(self, want):
        return all(torch().equal(a, b) for a, b in zip(self.results(), want))


SIZES = [dict(r=96, width=200, hidden=328), dict(r=2, width=1, hidden=1),
         dict(r=1200, width=640, hidden=2600, dtype="f16")]


@pytest.mark.parametrize("k", SIZES)
def test_strided_slices_and_other_streams(k):
    t = torch()
    say(f"[calls] {k}")
    A, B = Calls(1, **k), Calls(1, extra=64, **k)  # rows further apart
    A.run()
    t.cuda.synchronize()
    want = A.copy()
    B.run()
    t.cuda.synchronize()
    assert B.same(want), "strides"
    s = t.cuda.Stream()
    busy = t.randn(4096, 4096, device="cuda")
    for explicit in (True, False):
        A.wipe()
        s.wait_stream(t.cuda.current_stream())
        for _ in range(3):
            busy = busy @ busy * 1e-3  # the current stream is behind
        if explicit:
            A.run(stream=s)
        else:
            with t.cuda.stream(s):
                A.run()
        s.synchronize()
        assert A.same(want), f"stream, explicit {explicit}"
        t.cuda.synchronize()


@pytest.mark.parametrize("k", SIZES)
def test_two_at_once_and_again(k):
    t = torch()
    made = [Calls(s, **k) for s in (2, 3)]
    want = []
    for c in made:
        c.run()
        t.cuda.synchronize()
        want.append(c.copy())
        c.wipe()
    streams = [t.cuda.Stream() for _ in made]
    t.cuda.synchronize()
    for _ in range(4):
        for c, s in zip(made, streams):
            with t.cuda.stream(s):
                c.run()
    t.cuda.synchronize()
    assert all(c.same(w) for c, w in zip(made, want))


@pytest.mark.parametrize("k", SIZES)
def test_graphs_that_share_a_workspace(k):
    """Two captured runs on one workspace, replayed in turn with eager runs, other
    work and synchronisations between: every replay is the eager result."""
    t = torch()
    say(f"[calls] graphs {k}")
    A = Calls(4, **k)
    B = Calls(5, ws=A.ws, **k)
    want, graphs = [], []
    for c in (A, B):
        c.run()
        t.cuda.synchronize()
        want.append(c.copy())
        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        graph = t.cuda.CUDAGraph()
        with t.cuda.stream(side):
            with t.cuda.graph(graph, stream=side):
                c.run()
        t.cuda.synchronize()
        graphs.append(graph)
    for turn in range(4):
        for c, graph, w in zip((A, B), graphs, want):
            c.wipe()
            graph.replay()
            junk = t.randn(1 << 18, device="cuda").sum()
            if turn % 2:
                t.cuda.synchronize()
                assert c.same(w), turn
                c.run()
        t.cuda.synchronize()
        assert A.same(want[0]) and B.same(want[1]), turn
        del junk


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [512 * w - 37 * w for w in range(1, 17)] + [8193, 9000, 12321])
def test_rows_of_every_number_of_waves(c, dtype):
    """A row of a join does not depend on the others: 37 rows are the same as each
    by itself, forward and back; and the sums of the parameters' gradients are
    those of a single row's times one."""
    t = torch()
    g = gen(c)
    r = 37
    x, b, dz = (rows(g, r, c, dtype) for _ in range(3))
    p = {k: vec(g, c, k in ("gamma", "gamma_b", "gate"))
         for k in ("gamma", "beta", "gamma_b", "beta_b", "gate")}

    def run(i, j):
        m = j - i
        new = lambda: out_rows(m, c, dtype)[0]  # noqa: E731
        rr, z, dx, db = new(), new(), new(), new()
        rs = [t.zeros(m, device="cuda") for _ in range(2)]
        (q, e), (qb, eb) = oba.act8_buffers(m, c), oba.act8_buffers(m, c)
        oba.residual_norm(x[i:j], 1e-5, b=b[i:j], alpha=0.5, rstd_b=rs[1], qb=qb, eb=eb, r=rr,
                          z=z, rstd=rs[0], q=q, e=e, **p)
        grads = t.zeros((1, 5 * c), device="cuda")
        oba.residual_norm_backward(
            1, dx, grads, oba.residual_norm_backward_workspace(1, m, c), dz=dz[i:j], dr=x[i:j],
            alpha=0.5, q=q, e=e, rstd=rs[0], gamma=p["gamma"], at_gamma=0, at_beta=c, db=db,
            qb=qb, eb=eb, rstd_b=rs[1], gamma_b=p["gamma_b"], beta_b=p["beta_b"], gate=p["gate"],
            at_gate=2 * c, at_gamma_b=3 * c, at_beta_b=4 * c)
        return (rr, z, dx, db, *rs, q, e, qb, eb), grads

    whole, total = run(0, r)
    sums = t.zeros(5 * c, device="cuda", dtype=t.float64)
    size = t.zeros(5 * c, device="cuda", dtype=t.float64)
    for i in range(r):
        one, grads = run(i, i + 1)
        t.cuda.synchronize()
        for k, (a, v) in enumerate(zip(whole, one)):
            assert t.equal(a[i:i + 1], v), (i, k)
        sums += grads[0].double()
        size += grads[0].double().abs()
    # the gate's gradient is gamma_b S + beta_b T, with dgamma_b = gate S, dbeta_b = gate T
    size[2 * c:3 * c] = (size[3 * c:4 * c] * p["gamma_b"].abs()
                         + size[4 * c:] * p["beta_b"].abs()) / p["gate"].abs()
    # 37 additions in binary32 and each row's result's own rounding
    close(total[0], sums, 40 * UNIT * size + 1e-30, "sums")


def test_joins_past_32_bit_offsets():
    """2^31 elements are behind the last rows, which are those of a call of their own."""
    t = torch()
    say("[calls] large join")
    c, r, last = 8192, (1 << 18) + 40, 5
    g = gen(1)
    xs, bs = rows(g, last, c, "bf16"), rows(g, last, c, "bf16")
    p = {k: vec(g, c, k in ("gamma", "gamma_b", "gate"))
         for k in ("gamma", "beta", "gamma_b", "beta_b", "gate")}
    res = []
    for m in (r, last):
        x, b, o, z, dx, db = (t.zeros((m, c), device="cuda", dtype=t.bfloat16) for _ in range(6))
        x[-last:], b[-last:] = xs, bs
        rs = [t.zeros(m, device="cuda") for _ in range(2)]
        kept = oba.act8_buffers(m, c), oba.act8_buffers(m, c)
        oba.residual_norm(x, 1e-5, b=b, rstd_b=rs[1], qb=kept[1][0], eb=kept[1][1], r=o, z=z,
                          rstd=rs[0], q=kept[0][0], e=kept[0][1], kind="rms", **p)
        grads = t.zeros((1, 5 * c), device="cuda")
        oba.residual_norm_backward(  # z's gradient is z, r's is r
            1, dx, grads, oba.residual_norm_backward_workspace(1, m, c), dz=z, dr=o,
            q=kept[0][0], e=kept[0][1], rstd=rs[0], gamma=p["gamma"], at_gamma=0, at_beta=c,
            db=db, qb=kept[1][0], eb=kept[1][1], rstd_b=rs[1], gamma_b=p["gamma_b"],
            beta_b=p["beta_b"], gate=p["gate"], at_gate=2 * c, at_gamma_b=3 * c, at_beta_b=4 * c,
            kind="rms")
        t.cuda.synchronize()
        assert bool(t.isfinite(grads).all())
        res.append([v[-last:].clone() for v in (o, z, dx, db, *rs, *kept[0], *kept[1])])
        del x, b, o, z, dx, db, kept
    for k, (a, v) in enumerate(zip(*res)):
        assert t.equal(a, v), k


@pytest.mark.parametrize("k,dtype", [(128, "bf16"), (24, "f16")])
def test_gated_products_past_32_bit_offsets(k, dtype):
    """Results and kept forms of more than 2^31 elements: the last rows against the
    formula, in the kernels of many tiles and of few steps."""
    t = torch()
    say(f"[calls] large gated {k}")
    h, r, last = 2056, (1 << 20) + 300, 290
    g = gen(2)
    x = t.zeros((r, k), device="cuda", dtype=dt(dtype))
    x[-last:] = rows(g, last, k, dtype)
    w = rows(g, 2 * h, k, dtype, std=k ** -0.5)
    y = t.empty((r, h), device="cuda", dtype=dt(dtype))
    kept = [oba.act8_buffers(r, h) for _ in range(2)]
    oba.gated_linear(x, w, y, oba.gated_linear_workspace(r, k, h), qp=kept[0][0], ep=kept[0][1],
                     qu=kept[1][0], eu=kept[1][1])
    t.cuda.synchronize()
    xs, ws = x[-last:].double(), w.double()
    pu, err = xs @ ws.t(), (k + 2) * U * (xs.abs() @ ws.abs().t()) + 1e-30
    p, u, ep, eu = pu[:, :h], pu[:, h:], err[:, :h], err[:, h:]
    f = gate64(p, "silu")[0]
    ef = 1.13 * ep + gate_bounds(p, "silu")[0]
    ref = f * u
    ey = ef * u.abs() + eu * (f.abs() + ef) + UNIT * ref.abs()
    hb = half(dtype) * (1 + 2 ** -7)
    close(y[-last:], ref, ey + hb * ref.abs() + tiny(dtype) + 2.0 ** -120, "y")
    assert bool((y[:-last] == 0).all()), "rows of zeros"
    del y
    # back, from kept forms of their own in the last rows
    vals = []
    for q, e in kept:
        q.zero_()
        e.fill_(127)
        q8, e8, v = encode64(rows(g, last, h, "f32"))
        q[-last:], e[-last:] = q8, e8
        vals.append(v)
    w2 = rows(g, k, h, dtype, std=k ** -0.5)
    dpu = t.empty((r, 2 * h), device="cuda", dtype=dt(dtype))
    oba.gated_hidden_grad(x, w2, *kept[0], *kept[1], dpu,
                          oba.gated_hidden_grad_workspace(r, h, k))
    t.cuda.synchronize()
    w6 = w2.double()
    d, ed = xs @ w6, (k + 2) * U * (xs.abs() @ w6.abs()) + 1e-30
    f, df = gate64(vals[0], "silu")
    ef, edf = gate_bounds(vals[0], "silu")
    for got, a, ea in ((dpu[-last:, :h], df * vals[1], edf * vals[1].abs()),
                       (dpu[-last:, h:], f, ef)):
        ref = d * a
        e = ed * (a.abs() + ea) + d.abs() * ea + 2 * UNIT * ref.abs()
        close(got, ref, e + hb * ref.abs() + tiny(dtype) + 2.0 ** -120, "dpu")
