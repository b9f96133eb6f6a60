"""Cases of the gated feed-forward sub-layer's operators: what a training or a serving pass
computes there beside the linear layer's products.

Kinds of a case:
  gated        f(x wg^T + bg) * (x wu^T + bu), both projections' weights in one matrix; with
               keep8 both pre-activations and the result are kept in 8 bits too
  hidden_grad  the gradients of both pre-activations: with dh = dy w, dh * u * f'(p) and
               dh * f(p), p and u kept in 8 bits
  dropout      x / (1 - rate) where a counter-based generator's 16 bits say so, else 0, plus add
  join         r = alpha x + gate * dropout(norm(b)), z = norm(r): what lies between two blocks;
               with keep8 the normalised rows are kept in 8 bits
  join_grad    its backward pass for n workers of `rows` rows each: the gradients of x and b, and
               every worker's gradients of the parameters in its gradient row
"""
import math

import numpy
import torch

own = False

GROUP = 32
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
GATES = ["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"]
ETA = 1e-5
SITE = 5  # the dropout's number within a step


def listed():
    return [
        # one position through the gated projections at the width of the 48-layer transformer:
        # serving, the weights' bytes
        dict(name="gated_token", kind="gated", rows=1, n_in=1600, hidden=6400, dtype="bf16",
             gate="silu", bias=False, keep8=False),
        # a short odd batch, everything kept for its backward pass
        dict(name="gated_odd", kind="gated", rows=515, n_in=777, hidden=1001, dtype="f16",
             gate="gelu", bias=True, keep8=True),
        # a pre-training batch (128 sequences of 128 positions), everything kept in 8 bits
        dict(name="gated_batch", kind="gated", rows=16384, n_in=1024, hidden=4096, dtype="bf16",
             gate="silu", bias=True, keep8=True),
        # the short odd batch back through the second projection and the gate
        dict(name="hidden_grad_odd", kind="hidden_grad", rows=515, hidden=1001, n_out=777,
             dtype="f16", gate="gelu_tanh"),
        # the batch back
        dict(name="hidden_grad_batch", kind="hidden_grad", rows=16384, hidden=4096, n_out=1024,
             dtype="bf16", gate="silu"),
        # odd rows in binary32 with the stream they are added to
        dict(name="dropout_odd", kind="dropout", rows=4099, cols=1609, dtype="f32", rate=0.1,
             add=True),
        # a feed-forward's hidden activations of a batch
        dict(name="dropout_batch", kind="dropout", rows=32768, cols=4096, dtype="bf16", rate=0.1,
             add=False),
        # serving one position: nothing dropped, nothing kept; latency alone
        dict(name="join_token", kind="join", rows=1, cols=1600, dtype="bf16", norm="rms",
             pre=True, post=True, gate=True, beta=False, rate=0.0, alpha=1.0, keep8=False),
        # the join between two blocks of the batch with norms on both sides, all kept
        dict(name="join_batch", kind="join", rows=32768, cols=1024, dtype="bf16", norm="layer",
             pre=True, post=True, gate=True, beta=True, rate=0.1, alpha=1.25, keep8=True),
        # wide binary32 rows without a norm behind the block
        dict(name="join_wide", kind="join", rows=2048, cols=8192, dtype="f32", norm="rms",
             pre=True, post=False, gate=False, beta=False, rate=0.1, alpha=1.0, keep8=True),
        # odd numbers of workers, rows and columns, into binary32 gradient rows
        dict(name="join_grad_odd", kind="join_grad", n=3, rows=1001, cols=1111, dtype="f16",
             g="f32", norm="rms", pre=True, post=True, gate=True, beta=False, rate=0.2,
             alpha=0.75, dr=True),
        # the batch's backward pass, 8 workers, into 16-bit gradient rows
        dict(name="join_grad_batch", kind="join_grad", n=8, rows=4096, cols=1024, dtype="bf16",
             g="f16", norm="layer", pre=True, post=True, gate=True, beta=True, rate=0.1,
             alpha=1.25, dr=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["gated", "gated", "hidden_grad", "dropout", "join", "join", "join_grad",
                       "join_grad"])
    any_type = rng.choice(["f32", "f16", "bf16"])
    rate = rng.choice([0.0, 0.1, 0.3])
    if kind == "dropout":
        cols = _log(rng, 5, 9000)
        return dict(kind=kind, rows=_log(rng, 1, max(2, 60_000_000 // cols)), cols=cols,
                    dtype=any_type, rate=rate, add=rng.random() < 0.5)
    if kind in ("join", "join_grad"):
        cols = _log(rng, 24, 12000)
        post = rng.random() < 0.6
        c = dict(kind=kind, cols=cols, dtype=any_type, norm=rng.choice(["layer", "rms"]),
                 pre=rng.random() < 0.8, post=post, gate=rng.random() < 0.6,
                 beta=rng.random() < 0.5, rate=rate, alpha=rng.choice([1.0, 0.75, 2.5]))
        if kind == "join":
            return dict(c, rows=_log(rng, 1, max(2, 20_000_000 // cols)),
                        keep8=rng.random() < 0.6)
        n = rng.randint(1, 9)
        return dict(c, n=n, rows=_log(rng, 1, max(2, 20_000_000 // (cols * n))),
                    g=rng.choice(["f32", "f16", "bf16"]), dr=not c["pre"] or rng.random() < 0.7)
    two, gate = rng.choice(["f16", "bf16"]), rng.choice(GATES)
    wide, hidden = _log(rng, 24, 6500), _log(rng, 24, 6500)
    most = 90e9 / (4.0 * wide * hidden)  # rows that 90 GFLOP pay for
    rows = _log(rng, 1, max(2, min(16384, int(most))))
    if kind == "gated":
        return dict(kind=kind, rows=rows, n_in=wide, hidden=hidden, dtype=two, gate=gate,
                    bias=rng.random() < 0.5, keep8=rng.random() < 0.5)
    return dict(kind=kind, rows=rows, hidden=hidden, n_out=wide, dtype=two, gate=gate)


# ---- inputs -----------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _rows(gen, rows, cols, dtype, std):
    """[rows][cols] in a buffer whose row stride is a multiple of 8 elements; columns of
    different sizes, as a trained model's activations have them."""
    ld = (cols + 7) // 8 * 8
    t = torch.randn((rows, ld), generator=gen, device="cuda")
    t *= std * torch.exp(0.5 * torch.randn((1, ld), generator=gen, device="cuda"))
    return t.to(TYPES[dtype])[:, :cols]


def _like(rows, cols, dtype):
    ld = (cols + 7) // 8 * 8
    return torch.empty((rows, ld), dtype=TYPES[dtype], device="cuda")[:, :cols]


def _encode(x):
    """(q [rows][groups*32] int8, e [rows][groups] uint8): a group of largest magnitude
    f * 2^k, 1 <= f < 2, holds q = x / 2^(k-6) rounded to nearest even, at most 127 in
    magnitude; e = k - 6 + 127, at least 1."""
    rows, cols = x.shape
    groups = (cols + GROUP - 1) // GROUP
    p = torch.zeros((rows, groups * GROUP), device=x.device)
    p[:, :cols] = x.to(torch.float32)
    p = p.view(rows, groups, GROUP)
    top = p.abs().amax(dim=2)
    s = torch.clamp(torch.frexp(top)[1] - 7, min=-126)
    s = torch.where(top > 0, s, torch.full_like(s, -126))
    q = torch.clamp(torch.round(torch.ldexp(p, -s.unsqueeze(2))), -127, 127)
    return q.to(torch.int8).view(rows, groups * GROUP), (s + 127).to(torch.uint8)


def _decode(q, e, cols):
    rows, groups = e.shape
    s = torch.ldexp(torch.ones((), device=q.device), e.to(torch.int32) - 127)
    return (q.to(torch.float32).view(rows, groups, GROUP) * s.unsqueeze(2)).view(rows, -1)[:, :cols]


def _kept(rows, cols):
    groups = (cols + GROUP - 1) // GROUP
    return (torch.empty((rows, groups * GROUP), dtype=torch.int8, device="cuda"),
            torch.empty((rows, groups), dtype=torch.uint8, device="cuda"))


def _workspace(name, *sizes):
    """The workspace that a program makes once for these sizes; a tree without the operators
    has none to make."""
    try:
        from communication_compressed_optimizer_02_amd import binding as oba
        return getattr(oba, name)(*sizes)
    except (AttributeError, RuntimeError, OSError):
        return None


def _params(gen, c, s):
    """The join's parameters; None where it has none."""
    vec = lambda a, b: a + b * torch.randn(c["cols"], generator=gen, device="cuda")  # noqa: E731
    s["gamma"] = vec(1.0, 0.1) if c["pre"] else None
    s["beta"] = vec(0.0, 0.1) if c["pre"] and c["beta"] else None
    s["gamma_b"] = vec(1.0, 0.1) if c["post"] else None
    s["beta_b"] = vec(0.0, 0.1) if c["post"] and c["beta"] else None
    s["gate"] = vec(0.5, 0.2) if c["gate"] else None


def _needs_branch(c):
    """Whether the backward pass reads the branch: for its norm or for the gate's gradient."""
    return c["post"] or c["gate"]


def _places(c):
    """Offsets of the parameters' gradients in a gradient row, and its length."""
    names = (["gamma"] if c["pre"] else []) + (["beta"] if c["pre"] and c["beta"] else [])
    names += ["gate"] if c["gate"] else []
    names += (["gamma_b"] if c["post"] else []) + (["beta_b"] if c["post"] and c["beta"] else [])
    return {n: i * c["cols"] for i, n in enumerate(names)}, len(names) * c["cols"]


def prepare(case, seed):
    c, gen = dict(case), _gen(seed)
    k, t, dev = c["kind"], c["dtype"], "cuda"
    s = dict(case=c)
    # the dropout's seed and step, on the device: a captured step reads what is there
    s["rng"] = torch.tensor([(int(seed) * 0x9E3779B97F4A7C15 + 12345) % (1 << 63), int(seed) % 997],
                            dtype=torch.int64, device=dev)
    if k == "dropout":
        s["x"] = _rows(gen, c["rows"], c["cols"], t, 1.0)
        s["add"] = _rows(gen, c["rows"], c["cols"], t, 1.0) if c["add"] else None
        s["y"] = _like(c["rows"], c["cols"], t)
        return s
    if k == "join":
        rows, cols = c["rows"], c["cols"]
        s["x"], s["b"] = _rows(gen, rows, cols, t, 1.0), _rows(gen, rows, cols, t, 0.5)
        _params(gen, c, s)
        s["r"] = _like(rows, cols, t)
        if c["pre"]:
            s.update(z=_like(rows, cols, t), rstd=torch.empty(rows, device=dev))
        if c["post"]:
            s["rstd_b"] = torch.empty(rows, device=dev)
        if c["keep8"] and c["pre"]:
            s["q"], s["e"] = _kept(rows, cols)
            s["kept"] = _like(rows, cols, "bf16")
        if c["keep8"] and _needs_branch(c):
            s["qb"], s["eb"] = _kept(rows, cols)
            s["kept_b"] = _like(rows, cols, "bf16")
        return s
    if k == "join_grad":
        n, cols = c["n"], c["cols"]
        rows = n * c["rows"]
        _params(gen, c, s)
        s["dr"] = _rows(gen, rows, cols, t, 0.01) if c["dr"] else None
        if c["pre"]:
            s["dz"] = _rows(gen, rows, cols, t, 0.01)
            h, s["rstd"] = _normal(_rows(gen, rows, cols, t, 1.5).float(), c["norm"])
            s["q"], s["e"] = _encode(h)
        if _needs_branch(c):
            b = _rows(gen, rows, cols, t, 0.5).float()
            if c["post"]:
                b, s["rstd_b"] = _normal(b, c["norm"])
            s["qb"], s["eb"] = _encode(b)
        s["dx"], s["db"] = _like(rows, cols, t), _like(rows, cols, t)
        s["at"], size = _places(c)
        s["grads"] = torch.zeros((n, max(8, (size + 7) // 8 * 8)), dtype=TYPES[c["g"]], device=dev)
        s["ws"] = _workspace("residual_norm_backward_workspace", n, c["rows"], cols)
        return s
    rows, hidden = c["rows"], c["hidden"]
    if k == "gated":
        s["x"] = _rows(gen, rows, c["n_in"], t, 1.0)
        s["w"] = _rows(gen, 2 * hidden, c["n_in"], t, 0.02)
        s["bias"] = 0.1 * torch.randn(2 * hidden, generator=gen, device=dev) if c["bias"] else None
        s["y"] = _like(rows, hidden, t)
        if c["keep8"]:
            for name in "puy":
                s["q" + name], s["e" + name] = _kept(rows, hidden)
                s["kept_" + name] = _like(rows, hidden, "bf16")
        s["ws"] = _workspace("gated_linear_workspace", rows, c["n_in"], hidden)
        return s
    s["dy"] = _rows(gen, rows, c["n_out"], t, 0.01)
    s["w"] = _rows(gen, c["n_out"], hidden, t, 0.02)
    s["qp"], s["ep"] = _encode(_rows(gen, rows, hidden, t, 1.0))
    s["qu"], s["eu"] = _encode(_rows(gen, rows, hidden, t, 1.0))
    s["dpu"] = _like(rows, 2 * hidden, t)
    s["ws"] = _workspace("gated_hidden_grad_workspace", rows, hidden, c["n_out"])
    return s


# ---- the plain forms ---------------------------------------------------------------------

def _gate(p, kind):
    """f(p) and f'(p)."""
    if kind == "relu":
        return torch.clamp(p, min=0), (p > 0).to(p.dtype)
    if kind == "gelu":
        cdf = 0.5 * torch.erfc(-p * math.sqrt(0.5))
        return p * cdf, cdf + p * torch.exp(-0.5 * p * p) * (1 / math.sqrt(2 * math.pi))
    if kind == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (p + 0.044715 * p * p * p))
        du = math.sqrt(2 / math.pi) * (1.0 + 3 * 0.044715 * p * p)
        return 0.5 * p * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * p * (1.0 - t * t) * du
    if kind in ("silu", "sigmoid"):
        s = 1.0 / (1.0 + torch.exp(-p))
        g = s * (1.0 - s)
        return (p * s, s + p * g) if kind == "silu" else (s, g)
    return p, torch.ones_like(p)


def _normal(x, norm):
    """Normalised rows and the reciprocal of their spread."""
    if norm == "layer":
        x = x - x.mean(dim=1, keepdim=True)
    rstd = 1.0 / torch.sqrt((x * x).mean(dim=1) + ETA)
    return x * rstd[:, None], rstd


def _threshold(rate):
    return int(math.floor(rate * 65536 + 0.5))


def _keep(rng, rows, cols, rate):
    """Whether the 16 bits of an element reach the rate's share of 65536: Philox4x32-10 on
    (number of the eight columns' block in the matrix, site, step), its key the seed."""
    low = 0xFFFFFFFF
    blocks = (cols + 7) // 8
    i = torch.arange(rows * blocks, device=rng.device)
    c0, c1 = i & low, i >> 32
    c2, c3 = torch.full_like(i, SITE), (rng[1] & low).expand_as(i)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((b >> 32) & low) ^ c1 ^ k0, b & low,
                          ((a >> 32) & low) ^ c3 ^ k1, a & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    bits = torch.stack([h for w in (c0, c1, c2, c3) for h in (w & 0xFFFF, w >> 16)], dim=1)
    return (bits >= _threshold(rate)).view(rows, blocks * 8)[:, :cols]


def _drop(s, v, rate):
    if rate == 0:
        return v
    keep = _keep(s["rng"], v.shape[0], v.shape[1], rate)
    return torch.where(keep, v * (65536.0 / (65536 - _threshold(rate))), torch.zeros_like(v))


def _join(s, c):
    f, t = torch.float32, TYPES[c["dtype"]]
    out = {}
    v = s["b"].to(f)
    if c["post"]:
        v, out["rstd_b"] = _normal(v, c["norm"])
    if "kept_b" in s:
        out["kept_b"] = _decode(*_encode(v), c["cols"]).to(torch.bfloat16)
    if c["post"]:
        v = v * s["gamma_b"]
        if s["beta_b"] is not None:
            v = v + s["beta_b"]
    v = _drop(s, v, c["rate"])
    if c["gate"]:
        v = v * s["gate"]
    r = c["alpha"] * s["x"].to(f) + v
    out["r"] = r.to(t)
    if c["pre"]:
        h, out["rstd"] = _normal(r, c["norm"])
        if "kept" in s:
            out["kept"] = _decode(*_encode(h), c["cols"]).to(torch.bfloat16)
        z = h * s["gamma"]
        if s["beta"] is not None:
            z = z + s["beta"]
        out["z"] = z.to(t)
    return out


def _through(a, h, rstd, norm):
    """A norm's input gradient from that of its normalised rows."""
    d = a - h * (a * h).mean(dim=1, keepdim=True)
    if norm == "layer":
        d = d - a.mean(dim=1, keepdim=True)
    return d * rstd[:, None]


def _join_grad(s, c):
    f, t, cols = torch.float32, TYPES[c["dtype"]], c["cols"]
    per = lambda v: v.reshape(c["n"], -1, cols).sum(dim=1)  # noqa: E731
    grads = {}
    d = s["dr"].to(f) if c["dr"] else None
    if c["pre"]:
        dz, h = s["dz"].to(f), _decode(s["q"], s["e"], cols)
        grads["gamma"], grads["beta"] = per(dz * h), per(dz)
        through = _through(dz * s["gamma"], h, s["rstd"], c["norm"])
        d = through if d is None else through + d
    dx = c["alpha"] * d
    e = _drop(s, d, c["rate"])
    if _needs_branch(c):
        v = _decode(s["qb"], s["eb"], cols)
    if c["gate"]:
        whole = v * s["gamma_b"] if c["post"] else v
        if s["beta_b"] is not None:
            whole = whole + s["beta_b"]
        grads["gate"] = per(e * whole)
        e = e * s["gate"]
    if c["post"]:
        grads["gamma_b"], grads["beta_b"] = per(e * v), per(e)
        e = _through(e * s["gamma_b"], v, s["rstd_b"], c["norm"])
    out = dict(dx=dx.to(t), db=e.to(t))
    if s["at"]:
        out["g"] = torch.cat([grads[name] for name in s["at"]], dim=1).to(TYPES[c["g"]])
    return out


def _plain(s):
    c = s["case"]
    k, f, t = c["kind"], torch.float32, TYPES[c["dtype"]]
    if k == "dropout":
        y = _drop(s, s["x"].to(f), c["rate"])
        return dict(y=(y if s["add"] is None else y + s["add"].to(f)).to(t))
    if k == "join":
        return _join(s, c)
    if k == "join_grad":
        return _join_grad(s, c)
    hidden = c["hidden"]
    if k == "gated":
        pu = s["x"].to(f) @ s["w"].to(f).t()
        if s["bias"] is not None:
            pu = pu + s["bias"]
        p, u = pu[:, :hidden], pu[:, hidden:]
        y = (_gate(p, c["gate"])[0] * u).to(t)
        out = dict(y=y)
        if c["keep8"]:
            for name, v in (("p", p), ("u", u), ("y", y)):
                out["kept_" + name] = _decode(*_encode(v), hidden).to(torch.bfloat16)
        return out
    dh = s["dy"].to(f) @ s["w"].to(f)
    v, d = _gate(_decode(s["qp"], s["ep"], hidden), c["gate"])
    return dict(dpu=torch.cat([dh * _decode(s["qu"], s["eu"], hidden) * d, dh * v], dim=1).to(t))


# ---- the framework's calls ---------------------------------------------------------------

def _own(s):
    from communication_compressed_optimizer_02_amd import binding as oba
    c = s["case"]
    k = c["kind"]
    if k == "dropout":
        oba.dropout(s["x"], s["y"], s["rng"], c["rate"], site=SITE, add=s["add"])
        return dict(y=s["y"])
    if k == "join":
        oba.residual_norm(s["x"], ETA, b=s["b"], alpha=c["alpha"], gate=s["gate"],
                          gamma_b=s["gamma_b"], beta_b=s["beta_b"], rstd_b=s.get("rstd_b"),
                          qb=s.get("qb"), eb=s.get("eb"), rate=c["rate"], rng=s["rng"], site=SITE,
                          r=s["r"], gamma=s["gamma"], beta=s["beta"], z=s.get("z"),
                          rstd=s.get("rstd"), q=s.get("q"), e=s.get("e"), kind=c["norm"])
        out = {name: s[name] for name in ("rstd_b", "r", "rstd", "z") if name in s}
        for name, q, e in (("kept", "q", "e"), ("kept_b", "qb", "eb")):
            if name in s:
                oba.act8_decode(s[q], s[e], s[name])
                out[name] = s[name]
        return out
    if k == "join_grad":
        at = s["at"]
        oba.residual_norm_backward(
            c["n"], s["dx"], s["grads"], s["ws"], dz=s.get("dz"), dr=s["dr"], alpha=c["alpha"],
            q=s.get("q"), e=s.get("e"), rstd=s.get("rstd"), gamma=s["gamma"],
            at_gamma=at.get("gamma"), at_beta=at.get("beta"), db=s["db"], qb=s.get("qb"),
            eb=s.get("eb"), rstd_b=s.get("rstd_b"), gamma_b=s["gamma_b"], beta_b=s["beta_b"],
            gate=s["gate"], at_gate=at.get("gate"), at_gamma_b=at.get("gamma_b"),
            at_beta_b=at.get("beta_b"), rate=c["rate"], rng=s["rng"], site=SITE, kind=c["norm"])
        out = dict(dx=s["dx"], db=s["db"])
        if at:
            out["g"] = s["grads"][:, :len(at) * c["cols"]]
        return out
    if k == "gated":
        oba.gated_linear(s["x"], s["w"], s["y"], s["ws"], bias=s["bias"], gate=c["gate"],
                         qp=s.get("qp"), ep=s.get("ep"), qu=s.get("qu"), eu=s.get("eu"),
                         q=s.get("qy"), e=s.get("ey"))
        out = dict(y=s["y"])
        if c["keep8"]:
            for name in "puy":
                oba.act8_decode(s["q" + name], s["e" + name], s["kept_" + name])
                out["kept_" + name] = s["kept_" + name]
        return out
    oba.gated_hidden_grad(s["dy"], s["w"], s["qp"], s["ep"], s["qu"], s["eu"], s["dpu"], s["ws"],
                          gate=c["gate"])
    return dict(dpu=s["dpu"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -------------------------------------------------------

def work(case):
    c = case
    k, b = c["kind"], SIZE[c["dtype"]]
    kept = lambda r, w: r * ((w + GROUP - 1) // GROUP) * (GROUP + 1)  # noqa: E731
    if k == "dropout":
        return {"bytes": c["rows"] * c["cols"] * b * (3 if c["add"] else 2),
                "flops": 2 * c["rows"] * c["cols"]}
    if k in ("join", "join_grad"):
        r, w = c["rows"] * c.get("n", 1), c["cols"]
        branch = kept(r, w) if _needs_branch(c) else 0
        pre = kept(r, w) if c["pre"] else 0
        stats = 4 * r * (c["pre"] + c["post"])
        params = 4 * w * (c["gate"] + (c["pre"] + c["post"]) * (1 + c["beta"]))
        if k == "join":
            return {"bytes": r * w * b * (4 if c["pre"] else 3) + stats + params
                    + (branch + pre if c["keep8"] else 0),
                    "flops": r * w * (3 + 8 * (c["pre"] + c["post"]))}
        return {"bytes": r * w * b * (2 + c["pre"] + c["dr"]) + stats + params + branch + pre
                + c["n"] * _places(c)[1] * SIZE[c["g"]],
                "flops": r * w * (3 + 14 * (c["pre"] + c["post"]))}
    r, h = c["rows"], c["hidden"]
    if k == "gated":
        i = c["n_in"]
        return {"bytes": (r * i + 2 * h * i + r * h) * b + (8 * h if c["bias"] else 0)
                + (3 * kept(r, h) if c["keep8"] else 0), "flops": 4 * r * i * h}
    o = c["n_out"]
    return {"bytes": (r * o + o * h + 2 * r * h) * b + 2 * kept(r, h), "flops": 2 * r * o * h}


# ---- the definitions in 64 bits ----------------------------------------------------------

def _kept64(q, e, cols):
    steps = torch.pow(2.0, e.to(torch.float64) - 127.0).repeat_interleave(GROUP, dim=1)
    return (q.to(torch.float64) * steps)[:, :cols]


def _factor64(s, rows, cols, rate):
    """[rows][cols] of 0 and 1 / (1 - rate), the rate as a multiple of 2^-16: Philox4x32-10 in
    unsigned 64-bit integers on the host."""
    u = numpy.uint64
    mask, half = u(0xFFFFFFFF), u(32)
    seed, step = (int(v) for v in s["rng"].cpu())
    wide = -(-cols // 8)
    n = numpy.arange(rows * wide, dtype=u)
    x = [n & mask, n >> half, numpy.full_like(n, SITE), numpy.full_like(n, step % 2 ** 32)]
    key = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]
    for _ in range(10):
        first, second = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(second >> half) ^ x[1] ^ u(key[0]), second & mask,
             (first >> half) ^ x[3] ^ u(key[1]), first & mask]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    share = round(rate * 65536)
    kept = numpy.empty((rows * wide, 8), dtype=bool)
    for j in range(8):
        kept[:, j] = (x[j // 2] >> u(16 * (j % 2))) % u(65536) >= u(share)
    out = torch.from_numpy(kept.reshape(rows, wide * 8)[:, :cols].copy()).cuda()
    return out.to(torch.float64) / (1.0 - share / 65536)


def _gate64(p, kind):
    if kind == "relu":
        return p * (p > 0), (p > 0).to(p.dtype)
    if kind == "gelu":
        c = torch.special.ndtr(p)
        return p * c, c + p * torch.exp(-p ** 2 / 2) / math.sqrt(2 * math.pi)
    if kind == "none":
        return p, torch.ones_like(p)
    # p times the logistic function of a multiple of p or of p's cubic, or that function alone
    if kind == "gelu_tanh":
        a = math.sqrt(8 / math.pi)
        arg, darg = a * (p + 0.044715 * p ** 3), a * (1 + 3 * 0.044715 * p ** 2)
    else:
        arg, darg = p, torch.ones_like(p)
    s = torch.sigmoid(arg)
    slope = s * torch.sigmoid(-arg) * darg
    return (s, slope) if kind == "sigmoid" else (p * s, s + p * slope)


def _norm64(x, kind):
    z = x - x.mean(1, keepdim=True) if kind == "layer" else x
    rstd = (z.square().mean(1, keepdim=True) + ETA).rsqrt()
    return z * rstd, rstd


def _norm_grad64(dh, h, rstd, kind):
    n = h.shape[1]
    mean = dh.sum(1, keepdim=True) if kind == "layer" else 0.0
    return rstd.to(torch.float64)[:, None] / n * (n * dh - mean - h * (dh * h).sum(1, keepdim=True))


def exact(case, seed):
    s = prepare(case, seed)
    c, d = s["case"], torch.float64
    k = c["kind"]
    wide = lambda name: None if s.get(name) is None else s[name].to(d)  # noqa: E731
    if k == "dropout":
        y = wide("x") * _factor64(s, c["rows"], c["cols"], c["rate"])
        return dict(y=y + wide("add") if c["add"] else y)
    if k in ("join", "join_grad"):
        rows, cols = c["rows"] * c.get("n", 1), c["cols"]
        m = _factor64(s, rows, cols, c["rate"])
        gate = wide("gate") if c["gate"] else 1.0
        g_b = wide("gamma_b") if c["post"] else 1.0
        b_b = wide("beta_b") if s["beta_b"] is not None else 0.0
    if k == "join":
        out = {}
        v = wide("b")
        if c["post"]:
            v, rs = _norm64(v, c["norm"])
            out["rstd_b"] = rs[:, 0]
        if "kept_b" in s:
            out["kept_b"] = None  # next to a border the last bit of a sum says which integer
        out["r"] = r = c["alpha"] * wide("x") + gate * (m * (v * g_b + b_b))
        if c["pre"]:
            h, rs = _norm64(r, c["norm"])
            out["rstd"] = rs[:, 0]
            if "kept" in s:
                out["kept"] = None
            out["z"] = h * wide("gamma") + (wide("beta") if s["beta"] is not None else 0.0)
        return out
    if k == "join_grad":
        total = lambda v: v.reshape(c["n"], -1, cols).sum(1)  # noqa: E731
        gr, full = {}, 0.0
        if c["pre"]:
            h, dz = _kept64(s["q"], s["e"], cols), wide("dz")
            gr["gamma"], gr["beta"] = total(dz * h), total(dz)
            full = _norm_grad64(dz * wide("gamma"), h, s["rstd"], c["norm"])
        full = full + wide("dr") if c["dr"] else full
        dm = full * m
        if _needs_branch(c):
            v = _kept64(s["qb"], s["eb"], cols)
            gr["gate"] = total(dm * (v * g_b + b_b))
            gr["gamma_b"], gr["beta_b"] = total(dm * gate * v), total(dm * gate)
        db = dm * gate
        if c["post"]:
            db = _norm_grad64(db * g_b, v, s["rstd_b"], c["norm"])
        out = dict(dx=c["alpha"] * full, db=db)
        if s["at"]:
            out["g"] = torch.cat([gr[name] for name in s["at"]], dim=1)
        return out
    hidden, w = c["hidden"], wide("w")
    if k == "gated":
        p = torch.mm(wide("x"), w[:hidden].t().contiguous())
        u = torch.mm(wide("x"), w[hidden:].t().contiguous())
        if c["bias"]:
            p, u = p + wide("bias")[:hidden], u + wide("bias")[hidden:]
        out = dict(y=_gate64(p, c["gate"])[0] * u)
        return dict(out, kept_p=None, kept_u=None, kept_y=None) if c["keep8"] else out
    dh = torch.mm(wide("dy"), w)
    f, df = _gate64(_kept64(s["qp"], s["ep"], hidden), c["gate"])
    return dict(dpu=torch.cat([dh * _kept64(s["qu"], s["eu"], hidden) * df, dh * f], dim=1))
