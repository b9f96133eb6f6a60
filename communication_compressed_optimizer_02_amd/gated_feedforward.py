"""A stack of gated feed-forward sub-layers, trained by 1-bit Adam on n workers.

    z   = norm(r)
    h   = f(z wg^T + bg) * (z wu^T + bu)
    b   = h w2^T + b2
    r'  = alpha r + scale * dropout(norm_b(b))

for each of `layers` sub-layers, from r = x to y = the last r'.  norm and norm_b
are "layer" or "rms" norms; norm_b (post=True) and scale, one factor per column
(scale=True), are there when asked for.  One sub-layer's sum and the next one's
norm are one kernel.

The parameters are a range of the flat binary32 vector x of a State, the
gradients of the n workers go to the same range of its gradient rows g, and what
the backward pass needs is kept in 8 bits: the normalised rows, both products'
inputs, both pre-activations, and norm_b's rows (with post or scale).  Dropout
keeps no mask: its rows' bits come from rng = {seed, step} on the device, so add
1 to rng[1] after each step (in a captured step too).  An element's bits depend on
its row, its column and its sub-layer's number, counted from `site`: instances of
one seed that run in one step have sites of their own.  The rows of the workers
follow each other: worker i's are [i*rows, (i+1)*rows).

    F = GatedFeedForward(width, hidden, n, rows, layers=4, rate=0.1, seed=1)
    L = Layout(F.size, n, ...); S = State(L, "bf16")
    F.init(S.x)
    for step in ...:
        F.load(S.x)                  # 16-bit copies of the weights
        y = F.forward(x)             # x [n*rows][width]
        dx = F.backward(dy, S.g)     # every worker's gradients, in its row of g
        S.warmup(...)  or  S.step_deferred(...)
        F.rng[1] += 1

forward() keeps what the next backward() reads; infer() keeps nothing, drops
nothing and takes up to n*rows rows.  x and dy are not the instance's own y and
dx.  One instance serves one stream at a time, and so do all that share scratch
(share=, an instance of the same sizes), in captured graphs too.
"""
from __future__ import annotations

from . import binding as oba


# Products of few tiles split their sums and need a workspace: gated ones of at most 128
# tiles of 64 rows, linear ones of at most 256 tiles of 128 rows.
_SPLIT_ROWS = 256 * 128


def _product_bytes(rows, width, hidden):
    """The workspace of a forward pass's products for so many rows."""
    c = oba.lib()
    return max(c.oba_gated_linear_workspace_bytes(rows, width, hidden),
               c.oba_linear_workspace_bytes(rows, hidden, width))


def _hungriest(width, hidden, total):
    """The number of rows up to total whose products need the largest workspace: fewer
    rows, split more often, may need more.  Of the counts between two multiples of 64,
    whose tiles are the same, the last needs the most."""
    counts = {min(m, total) for m in range(64, min(total, _SPLIT_ROWS) + 64, 64)} | {total}
    return max(counts, key=lambda m: _product_bytes(m, width, hidden))


class GatedFeedForward:
    def __init__(self, width, hidden, n, rows, layers=1, dtype="bf16", gate="silu", norm="rms",
                 eta=1e-5, alpha=1.0, rate=0.0, seed=0, site=0, post=False, scale=False,
                 at=0, share=None):
        import torch

        if gate not in oba.GATES:
            raise ValueError(f"gate: {gate!r} is none of {sorted(oba.GATES)}")
        if norm not in oba.NORMS:
            raise ValueError(f"norm: {norm!r} is none of {sorted(oba.NORMS)}")
        if layers < 1:
            raise ValueError(f"layers: {layers}")
        types = {"f16": torch.float16, "bf16": torch.bfloat16}
        if dtype not in types:
            raise ValueError(f"dtype: {dtype!r} is none of {sorted(types)}")
        sizes = (width, hidden, n, rows, types[dtype], torch.cuda.current_device())
        if share is not None and share.sizes != sizes:
            raise ValueError(f"share: an instance of {share.sizes}, not of {sizes}")
        self.sizes = sizes
        self.width, self.hidden, self.n, self.rows, self.layers = width, hidden, n, rows, layers
        self.gate, self.norm, self.eta, self.alpha, self.rate = gate, norm, eta, alpha, rate
        self.site, self.post, self.scale = site, post, scale
        self.flat = None  # the parameters that load() was given
        self.kept = False  # whether a forward() has left what backward() reads
        self.dtype = sizes[4]
        self.rng = oba.dropout_rng(seed)
        # the parameters' places in the flat vector, from `at`
        names = [("gamma", width)] + [("beta", width)] * (norm == "layer")
        names += [("w1", 2 * hidden * width), ("b1", 2 * hidden), ("w2", width * hidden),
                  ("b2", width)]
        if post:
            names += [("gamma_b", width)] + [("beta_b", width)] * (norm == "layer")
        names += [("scale", width)] * scale
        self.places, pos = [], at
        for _ in range(layers):
            place = {}
            for name, length in names:
                place[name] = (pos, length)
                pos += length
            self.places.append(place)
        self.size = pos - at
        total = n * rows

        def matrix(r, c):
            return torch.empty((r, (c + 7) // 8 * 8), dtype=self.dtype, device="cuda")[:, :c]

        def each(make):
            return [make() for _ in range(layers)]

        self.w1 = each(lambda: matrix(2 * hidden, width))
        self.w2 = each(lambda: matrix(width, hidden))
        self.y, self.dx = matrix(total, width), matrix(total, width)
        self.rstd = each(lambda: torch.empty(total, device="cuda"))
        self.kept_norm = each(lambda: oba.act8_buffers(total, width))  # norm(r)
        self.kept_z = each(lambda: oba.act8_buffers(total, width))  # the gated product's input
        self.kept_p = each(lambda: oba.act8_buffers(total, hidden))  # its two halves
        self.kept_u = each(lambda: oba.act8_buffers(total, hidden))
        self.kept_h = each(lambda: oba.act8_buffers(total, hidden))  # the second one's input
        if post:
            self.rstd_b = each(lambda: torch.empty(total, device="cuda"))
        if post or scale:
            self.kept_b = each(lambda: oba.act8_buffers(total, width))
        if share is not None:
            self.z, self.h, self.b, self.r = share.z, share.h, share.b, share.r
            self.dpu, self.dz, self.db, self.ws = share.dpu, share.dz, share.db, share.ws
            self.spare = share.spare
            return
        self.z, self.h, self.b = matrix(total, width), matrix(total, hidden), matrix(total, width)
        self.r = [matrix(total, width) for _ in range(2)]  # r, and its gradients
        self.spare = [torch.empty(total, device="cuda") for _ in range(2)]  # infer()'s rstd
        self.dpu, self.dz, self.db = (matrix(total, c) for c in (2 * hidden, width, width))
        self.ws = max((self._infer_workspace(total),
                       oba.gated_hidden_grad_workspace(total, hidden, width),
                       oba.linear_workspace(total, width, 2 * hidden),
                       oba.linear_weight_grad_workspace(n, rows, width, 2 * hidden),
                       oba.linear_weight_grad_workspace(n, rows, hidden, width),
                       oba.residual_norm_backward_workspace(n, rows, width)),
                      key=lambda t: t.numel())

    def _infer_workspace(self, total):
        """For every number of rows up to total."""
        at = _hungriest(self.width, self.hidden, total)
        return max((oba.gated_linear_workspace(at, self.width, self.hidden),
                    oba.linear_workspace(at, self.hidden, self.width)), key=lambda t: t.numel())

    def part(self, flat, layer, name):
        """A parameter's slice of the flat vector (or of a row of g)."""
        at, length = self.places[layer][name]
        return flat[at:at + length]

    def init(self, flat, generator=None):
        """Norms' gains and scales 1, biases 0, weights N(0, 1/inputs) (w2 halved)."""
        for layer, place in enumerate(self.places):
            for name in place:
                p = self.part(flat, layer, name)
                if name == "w1":
                    p.normal_(0.0, self.width ** -0.5, generator=generator)
                elif name == "w2":
                    p.normal_(0.0, 0.5 * self.hidden ** -0.5, generator=generator)
                else:
                    p.fill_(1.0 if name in ("gamma", "gamma_b", "scale") else 0.0)

    def load(self, flat):
        """The 16-bit copies of the weights, after every step of the optimizer."""
        self.flat = flat
        for k in range(self.layers):
            self.w1[k].copy_(self.part(flat, k, "w1").view(2 * self.hidden, self.width))
            self.w2[k].copy_(self.part(flat, k, "w2").view(self.width, self.hidden))

    def _opt(self, layer, name):
        return self.part(self.flat, layer, name) if name in self.places[layer] else None

    def _join(self, layer):
        """Sub-layer `layer`'s sum's parameters."""
        return dict(alpha=self.alpha, gate=self._opt(layer, "scale"),
                    gamma_b=self._opt(layer, "gamma_b"), beta_b=self._opt(layer, "beta_b"),
                    site=self.site + layer)

    def _next(self, layer, z, keep, m):
        """The norm of sub-layer `layer`."""
        q, e = self.kept_norm[layer] if keep else (None, None)
        return dict(gamma=self.part(self.flat, layer, "gamma"), beta=self._opt(layer, "beta"), z=z,
                    rstd=self.rstd[layer] if keep else self.spare[0][:m], q=q, e=e)

    def _pass(self, x, keep):
        if self.flat is None:
            raise RuntimeError("load() the parameters first")
        m, last = x.shape[0], self.layers - 1
        z, h, b, y = self.z[:m], self.h[:m], self.b[:m], self.y[:m]
        oba.residual_norm(x, self.eta, kind=self.norm, **self._next(0, z, keep, m))
        r = x
        for k in range(self.layers):
            kept = {}
            if keep:
                oba.act8_encode(z, *self.kept_z[k])
                for name, of in (("p", self.kept_p), ("u", self.kept_u), ("", self.kept_h)):
                    kept["q" + name], kept["e" + name] = of[k]
            oba.gated_linear(z, self.w1[k], h, self.ws, bias=self.part(self.flat, k, "b1"),
                             gate=self.gate, **kept)
            oba.linear(h, self.w2[k], b, self.ws, bias=self.part(self.flat, k, "b2"))
            join = self._join(k)
            if self.post:
                join["rstd_b"] = self.rstd_b[k] if keep else self.spare[1][:m]
            if keep:
                join.update(rate=self.rate, rng=self.rng)
                if self.post or self.scale:
                    join["qb"], join["eb"] = self.kept_b[k]
            if k < last:
                join.update(self._next(k + 1, z, keep, m))
            out = y if k == last else self.r[k % 2][:m]
            oba.residual_norm(r, self.eta, b=b, r=out, kind=self.norm, **join)
            r = out
        return y

    def forward(self, x):
        """y, in a buffer of the instance that the next forward() or infer()
        overwrites."""
        if x.shape[0] != self.n * self.rows:
            raise ValueError(f"x: {x.shape[0]} rows, not {self.n} x {self.rows}")
        y = self._pass(x, True)
        self.kept = True
        return y

    def infer(self, x):
        """y of up to n*rows rows, without dropout; what forward() kept stays."""
        if x.shape[0] > self.n * self.rows:
            raise ValueError(f"x: {x.shape[0]} rows, more than {self.n} x {self.rows}")
        return self._pass(x, False)

    def backward(self, dy, g):
        """dx (in a buffer of the instance), and every worker's gradients in its
        row of g [n][ld].  rng[1] is still the forward pass's."""
        if not self.kept:
            raise RuntimeError("forward() first: there is nothing kept to read")
        dr, n = dy, self.n
        for k in range(self.layers - 1, -1, -1):
            at = {name: place[0] for name, place in self.places[k].items()}
            back = self._join(k)
            if self.post:
                back["rstd_b"] = self.rstd_b[k]
            if self.post or self.scale:
                back["qb"], back["eb"] = self.kept_b[k]
            back.update(at_gate=at.get("scale"), at_gamma_b=at.get("gamma_b"),
                        at_beta_b=at.get("beta_b"), rate=self.rate, rng=self.rng)
            if k < self.layers - 1:
                back.update(self._norm(k + 1))
            out = self.r[k % 2]
            oba.residual_norm_backward(n, out, g, self.ws, dr=dr, db=self.db, kind=self.norm,
                                       **back)
            dr = out
            oba.linear_weight_grad(n, self.db, *self.kept_h[k], g, self.hidden, at["w2"],
                                   at["b2"], self.ws)
            oba.gated_hidden_grad(self.db, self.w2[k], *self.kept_p[k], *self.kept_u[k], self.dpu,
                                  self.ws, gate=self.gate)
            oba.linear_weight_grad(n, self.dpu, *self.kept_z[k], g, self.width, at["w1"],
                                   at["b1"], self.ws)
            oba.linear_input_grad(self.dpu, self.w1[k], self.dz, self.ws)
        oba.residual_norm_backward(n, self.dx, g, self.ws, dr=dr, kind=self.norm, **self._norm(0))
        return self.dx

    def _norm(self, layer):
        """What the gradient of sub-layer `layer`'s norm is made of."""
        place = self.places[layer]
        q, e = self.kept_norm[layer]
        return dict(dz=self.dz, q=q, e=e, rstd=self.rstd[layer],
                    gamma=self.part(self.flat, layer, "gamma"), at_gamma=place["gamma"][0],
                    at_beta=place["beta"][0] if "beta" in place else None)
