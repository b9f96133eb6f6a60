"""What is dropped is 0, whatever it was: rows of a join whose branch (or whose
gradient) is not finite, all of it dropped, are as if it had been finite.  The lanes
hold more columns than the row, and the rates drop some of the rows whole."""
import pytest

from communication_compressed_optimizer_02_amd import binding as oba
from layer_common import gen, out_rows, rows, torch
from sublayer_common import factor_gpu

pytestmark = pytest.mark.gpu

# columns, and the power of two that is kept: rows of less than a wave, of two waves, and of
# the form of 16 columns a lane
SIZES = [(1, 3), (2, 3), (3, 3), (5, 3), (8, 3), (11, 3), (600, 8), (8200, 13)]
SEED, STEP, SITE, ROWS = 77, 3, 2, 200


def vec(g, c):
    return 1.0 + 0.1 * torch().randn(c, generator=g, device="cuda")


def dropped(c, rate):
    """Whether all of a row is dropped: some are, some are not."""
    gone = (factor_gpu(ROWS, c, rate, SEED, STEP, SITE) == 0).all(1)
    assert bool(gone.any()) and not bool(gone.all())
    return gone


def same(a, b):
    return bool((a == b).all())


@pytest.mark.parametrize("branch", ["nan", "infinity", "zero"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("c,share", SIZES)
def test_forward(c, share, dtype, kind, branch):
    """A branch with a NaN or an infinity in each row, or of zeros without eta."""
    t, rate = torch(), 1 - 2.0 ** -share
    g = gen(c)
    x, b = rows(g, ROWS, c, dtype), rows(g, ROWS, c, dtype)
    p = {k: vec(g, c) for k in ("gamma", "beta", "gamma_b", "beta_b", "gate")}
    if c == 1 and kind == "layer":
        kind = "rms"  # a column's own mean leaves 0
    eta = 0.0 if branch == "zero" else 1e-5
    bad = b.clone()
    if branch == "zero":
        bad.zero_()
    else:
        bad[:, 0] = float("nan" if branch == "nan" else "inf")
    whole = t.empty((ROWS, (c + 7) // 8 * 8), device="cuda", dtype=x.dtype)
    whole[:, :c] = bad
    res = []
    for v in (b, whole[:, :c]):
        r, z = out_rows(ROWS, c, dtype)[0], out_rows(ROWS, c, dtype)[0]
        rstd, rstd_b = t.zeros(ROWS, device="cuda"), t.zeros(ROWS, device="cuda")
        q, e = oba.act8_buffers(ROWS, c)
        oba.residual_norm(x, eta, b=v, alpha=0.5, rstd_b=rstd_b, rate=rate,
                          rng=t.tensor([SEED, STEP], device="cuda"), site=SITE, r=r, z=z,
                          rstd=rstd, q=q, e=e, kind=kind, **p)
        t.cuda.synchronize()
        res.append((r, z, rstd, q, e))
    gone = dropped(c, rate)
    assert bool(t.isfinite(res[0][1][gone].float()).all())
    assert same(res[1][0][gone], 0.5 * x[gone])
    for k, (a, v) in enumerate(zip(*res)):
        assert same(a[gone], v[gone]), k
    if branch != "infinity":  # of an infinity the RMS norm leaves 0 in the other columns
        assert bool((~t.isfinite(res[1][1][~gone].float())).all(1).all())


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("c,share", SIZES)
def test_backward(c, share, dtype, kind, gated):
    """z's gradient has an infinity in each row, so that r's is not finite; the
    branch's is 0 where all of it is dropped."""
    t, rate = torch(), 1 - 2.0 ** -share
    g = gen(c + 50)
    dz = rows(g, ROWS, c, dtype)
    dz[:, 0] = float("inf")
    p = {k: vec(g, c) for k in ("gamma", "gamma_b")}
    if gated:
        p["gate"] = vec(g, c)
    (q, e), (qb, eb) = oba.act8_buffers(ROWS, c), oba.act8_buffers(ROWS, c)
    for kept in ((q, e), (qb, eb)):
        oba.act8_encode(rows(g, ROWS, c, dtype), *kept)
    dx, db = out_rows(ROWS, c, dtype)[0], out_rows(ROWS, c, dtype)[0]
    rstd, rstd_b = (t.ones(ROWS, device="cuda") for _ in range(2))
    oba.residual_norm_backward(1, dx, None, None, dz=dz, q=q, e=e, rstd=rstd, db=db, qb=qb, eb=eb,
                               rstd_b=rstd_b, rate=rate, rng=t.tensor([SEED, STEP], device="cuda"),
                               site=SITE, kind=kind, **p)
    t.cuda.synchronize()
    gone = dropped(c, rate)
    assert bool((db[gone] == 0).all())
    assert bool((~t.isfinite(dx.float())).any(1).all())
