"""A transformer's feed-forward sub-layer, trained by 1-bit Adam on n workers.

    y = x + act(norm(x) w1^T + b1) w2^T + b2

The parameters are a range of the flat binary32 vector x of a State, the
gradients of the n workers go to the same range of its gradient rows g, and
what the backward pass needs is kept in 8 bits: the normalised rows, both
products' inputs and the pre-activation, 2 1/16 bytes per row and column of
width and of hidden where 16-bit copies take 4.  Beside these an instance holds
its results y and dx (4 bytes per row and column of width), rstd and the 16-bit
copies of the weights.  The 16-bit rows that live within one pass (4 bytes per
row and column of width and of hidden) and the workspace are scratch: the layers
of a stack hold them once if each is made with share=, an instance of the same
sizes.  The rows of the workers follow each other: worker
i's are [i*rows, (i+1)*rows).

    F = FeedForward(width, hidden, n, rows)
    L = Layout(F.size, n, ...); S = State(L, "bf16")
    F.init(S.x)
    for step in ...:
        F.load(S.x)                  # 16-bit copies of the weights
        y = F.forward(x)             # x [n*rows][width]
        dx = F.backward(dy, S.g)     # every worker's gradients, in its row of g
        S.warmup(...)  or  S.step_deferred(...)

forward() keeps what the next backward() reads; x itself is read by forward()
only.  x and dy are not the instance's own y and dx.  One instance serves one
stream at a time, and so do all that share scratch, in captured graphs too.
"""
from __future__ import annotations

from . import binding as oba


class FeedForward:
    def __init__(self, width, hidden, n, rows, dtype="bf16", act="gelu", eta=1e-5, at=0,
                 share=None):
        import torch

        if act not in oba.ACTS:
            raise ValueError(f"act: {act!r} is none of {sorted(oba.ACTS)}")
        sizes = (width, hidden, n, rows, {"f16": torch.float16, "bf16": torch.bfloat16}[dtype],
                 torch.cuda.current_device())
        if share is not None and share.sizes != sizes:
            raise ValueError(f"share: an instance of {share.sizes}, not of {sizes}")
        self.sizes = sizes
        self.width, self.hidden, self.n, self.rows = width, hidden, n, rows
        self.act, self.eta = act, eta
        self.flat = None  # the parameters that load() was given
        self.kept = False  # whether a forward() has left what backward() reads
        self.dtype = sizes[4]
        # the parameters' places in the flat vector, from `at`
        self.places, pos = {}, at
        for name, length in (("gamma", width), ("beta", width), ("w1", hidden * width),
                             ("b1", hidden), ("w2", width * hidden), ("b2", width)):
            self.places[name] = (pos, length)
            pos += length
        self.size = pos - at
        total = n * rows

        def matrix(r, c):
            return torch.empty((r, (c + 7) // 8 * 8), dtype=self.dtype, device="cuda")[:, :c]

        self.w1, self.w2 = matrix(hidden, width), matrix(width, hidden)
        self.y, self.dx = matrix(total, width), matrix(total, width)
        self.rstd = torch.empty(total, device="cuda")
        self.kept_norm = oba.act8_buffers(total, width)   # xhat
        self.kept_z = oba.act8_buffers(total, width)      # the first product's input
        self.kept_pre = oba.act8_buffers(total, hidden)   # its result before act
        self.kept_h = oba.act8_buffers(total, hidden)     # the second product's input
        if share is not None:
            self.z, self.h, self.dz, self.dh = share.z, share.h, share.dz, share.dh
            self.mean, self.ws = share.mean, share.ws
            return
        self.z, self.h = matrix(total, width), matrix(total, hidden)
        self.dz, self.dh = matrix(total, width), matrix(total, hidden)
        self.mean = torch.empty(total, device="cuda")
        self.ws = max((oba.linear_workspace(total, width, hidden),
                       oba.linear_workspace(total, hidden, width),
                       oba.linear_weight_grad_workspace(n, rows, width, hidden),
                       oba.linear_weight_grad_workspace(n, rows, hidden, width),
                       oba.layer_norm_backward_workspace(n, rows, width)),
                      key=lambda t: t.numel())

    def part(self, flat, name):
        """A parameter's slice of the flat vector (or of a row of g)."""
        at, length = self.places[name]
        return flat[at:at + length]

    def init(self, flat, generator=None):
        """gamma 1, biases 0, weights N(0, 1/inputs) (w2 halved), in place."""
        for name, std in (("w1", self.width ** -0.5), ("w2", 0.5 * self.hidden ** -0.5)):
            self.part(flat, name).normal_(0.0, std, generator=generator)
        self.part(flat, "gamma").fill_(1.0)
        for name in ("beta", "b1", "b2"):
            self.part(flat, name).zero_()

    def load(self, flat):
        """The 16-bit copies of the weights, after every step of the optimizer."""
        self.flat = flat
        self.w1.copy_(self.part(flat, "w1").view(self.hidden, self.width))
        self.w2.copy_(self.part(flat, "w2").view(self.width, self.hidden))

    def forward(self, x):
        """y, in a buffer of the instance that the next forward() overwrites."""
        p = self.flat
        if p is None:
            raise RuntimeError("load() the parameters first")
        oba.layer_norm(x, self.part(p, "gamma"), self.part(p, "beta"), self.eta, self.z,
                       self.mean, self.rstd, *self.kept_norm)
        oba.act8_encode(self.z, *self.kept_z)
        oba.linear(self.z, self.w1, self.h, self.ws, bias=self.part(p, "b1"), act=self.act,
                   q=None if self.act == "none" else self.kept_pre[0],
                   e=None if self.act == "none" else self.kept_pre[1])
        oba.act8_encode(self.h, *self.kept_h)
        oba.linear(self.h, self.w2, self.y, self.ws, bias=self.part(p, "b2"), residual=x)
        self.kept = True
        return self.y

    def backward(self, dy, g):
        """dx (in a buffer of the instance), and every worker's gradients in its
        row of g [n][ld]."""
        if not self.kept:
            raise RuntimeError("forward() first: there is nothing kept to read")
        at = {name: place[0] for name, place in self.places.items()}
        pre = (None, None) if self.act == "none" else self.kept_pre
        oba.linear_weight_grad(self.n, dy, *self.kept_h, g, self.hidden, at["w2"], at["b2"],
                               self.ws)
        oba.linear_input_grad(dy, self.w2, self.dh, self.ws, act=self.act, q=pre[0], e=pre[1])
        oba.linear_weight_grad(self.n, self.dh, *self.kept_z, g, self.width, at["w1"], at["b1"],
                               self.ws)
        oba.linear_input_grad(self.dh, self.w1, self.dz, self.ws)
        oba.layer_norm_backward(self.n, self.dz, self.part(self.flat, "gamma"), self.rstd,
                                self.dx, g, at["gamma"], at["beta"], self.ws,
                                q=self.kept_norm[0], e=self.kept_norm[1], add=dy)
        return self.dx
