"""Refusals of the gated feed-forward sub-layer's operators: argument errors are
found on the host, before any HIP call, so made-up addresses serve and nothing is
launched.  They run where there is no GPU: a refusal that is missing ends in a
failed launch."""
import ctypes
import os

import pytest

from communication_compressed_optimizer_02_amd import binding as oba

no_gpu = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                            reason="made-up addresses: not where a GPU could read them")

EINVAL, EALIGN, EWORKSPACE, EHIP = -1, -2, -4, -5
F32, F16, BF16 = 0, 1, 2
A = 0x1000  # an aligned address that no call may touch
NAN, INF = float("nan"), float("inf")


def call(name, base, **change):
    """The entry point with base's arguments (in order), some changed."""
    args = dict(base)
    assert set(change) <= set(args), set(change) - set(args)
    args.update(change)
    fn = getattr(oba.lib(), name)
    return fn(*[ctypes.c_void_p(v) if t is ctypes.c_void_p else v
                for v, t in zip(args.values(), fn.argtypes)])


DROP = dict(rows=4, cols=40, x=A, ldx=40, dtype=BF16, rate=0.1, rng=A, site=1, add=A, ldadd=40,
            y=A, ldy=40, stream=None)
JOIN = dict(rows=4, cols=40, dtype=BF16, kind=0, eta=1e-5, x=A, ldx=40, alpha=1.0, b=A, ldb=40,
            gamma_b=A, beta_b=A, gate=A, rate=0.1, rng=A, site=0, rstd_b=A, qb=A, eb=A, r=A,
            ldr=40, gamma=A, beta=A, z=A, ldz=40, rstd=A, q=A, e=A, stream=None)
BACK = dict(n=2, rows=4, cols=40, dtype=BF16, kind=1, dz=A, lddz=40, q=A, e=A, rstd=A, gamma=A,
            dr=A, lddr=40, alpha=1.0, dx=A, lddx=40, qb=A, eb=A, rstd_b=A, gamma_b=A, beta_b=A,
            gate=A, rate=0.1, rng=A, site=0, db=A, lddb=40, dgamma=A, dbeta=A, dgamma_b=A,
            dbeta_b=A, dgate=A, g_dtype=F16, ldg=200, ws=A, ws_bytes=1 << 20, stream=None)
GATED = dict(rows=100, n_in=2048, hidden=64, x=A, ldx=2048, w=A, ldw=2048, dtype=BF16, bias=A,
             gate=4, y=A, ldy=64, qp=A, ep=A, qu=A, eu=A, q=A, e=A, ws=A, ws_bytes=1 << 26,
             stream=None)
GRAD = dict(rows=100, hidden=64, n_out=2048, dy=A, lddy=2048, w=A, ldw=64, dtype=F16, gate=4, qp=A,
            ep=A, qu=A, eu=A, dpu=A, lddpu=128, ws=A, ws_bytes=1 << 26, stream=None)
NO_BRANCH = dict(b=None, gamma_b=None, beta_b=None, gate=None, rate=0.0, rng=None, rstd_b=None,
                 qb=None, eb=None)
NO_NORM = dict(gamma=None, beta=None, z=None, rstd=None, q=None, e=None)
NO_DZ = dict(dz=None, q=None, e=None, rstd=None, gamma=None, dgamma=None, dbeta=None)
BASES = {"oba_dropout": DROP, "oba_residual_norm": JOIN, "oba_residual_norm_backward": BACK,
         "oba_gated_linear": GATED, "oba_gated_hidden_grad": GRAD}

CASES = {
    "oba_dropout": [
        (dict(rows=-1), EINVAL), (dict(rows=(1 << 30) + 1), EINVAL), (dict(cols=0), EINVAL),
        (dict(cols=(1 << 20) + 1, ldx=1 << 21, ldy=1 << 21, ldadd=1 << 21), EINVAL),
        (dict(ldx=32), EINVAL), (dict(ldy=44), EINVAL), (dict(ldadd=32), EINVAL),
        (dict(dtype=3), EINVAL), (dict(rate=-0.1), EINVAL), (dict(rate=1.0), EINVAL),
        (dict(rate=NAN), EINVAL), (dict(rate=INF), EINVAL), (dict(rate=1.0 - 2.0 ** -18), EINVAL),
        (dict(x=None), EINVAL), (dict(y=None), EINVAL), (dict(rng=None), EINVAL),
        (dict(x=A + 8), EALIGN), (dict(y=A + 4), EALIGN), (dict(add=A + 2), EALIGN),
        (dict(rng=A + 4), EALIGN),
        (dict(rows=1 << 30, cols=1 << 13, ldx=1 << 13, ldy=1 << 13, add=None), EINVAL)],
    "oba_residual_norm": [
        (dict(rows=-1), EINVAL), (dict(cols=0), EINVAL),
        (dict(cols=16385, ldx=16392, ldb=16392, ldr=16392, ldz=16392), EINVAL),
        (dict(ldx=32), EINVAL), (dict(ldb=41), EINVAL), (dict(ldr=8), EINVAL),
        (dict(ldz=8), EINVAL), (dict(dtype=3), EINVAL), (dict(kind=2), EINVAL),
        (dict(kind=-1), EINVAL), (dict(eta=-1.0), EINVAL), (dict(eta=NAN), EINVAL),
        (dict(alpha=INF), EINVAL), (dict(alpha=NAN), EINVAL), (dict(rate=1.0), EINVAL),
        (dict(alpha=1e39), EINVAL), (dict(eta=1e39), EINVAL),
        (dict(rate=-1e-9), EINVAL), (dict(x=None), EINVAL), (dict(x=A + 8), EALIGN),
        (dict(b=None), EINVAL), (dict(b=A + 8), EALIGN), (dict(gamma_b=None), EINVAL),
        (dict(gamma_b=None, beta_b=None), EINVAL), (dict(rstd_b=None), EINVAL),
        (dict(gamma_b=A + 2), EALIGN), (dict(beta_b=A + 1), EALIGN), (dict(gate=A + 2), EALIGN),
        (dict(qb=None), EINVAL), (dict(eb=None), EINVAL), (dict(qb=A + 8), EALIGN),
        (dict(rng=None), EINVAL), (dict(rng=A + 4), EALIGN), (dict(r=A + 8), EALIGN),
        (dict(gamma=None), EINVAL), (dict(z=None), EINVAL), (dict(rstd=None), EINVAL),
        (dict(z=A + 2), EALIGN), (dict(beta=A + 2), EALIGN), (dict(q=None), EINVAL),
        (dict(e=None), EINVAL), (dict(q=A + 4), EALIGN), (dict(r=None, **NO_NORM), EINVAL)]
    + [(dict({**NO_BRANCH, k: A}), EINVAL) for k in ("gamma_b", "beta_b", "gate", "rstd_b", "qb",
                                                     "eb")]
    + [(dict(NO_BRANCH, rate=0.1, rng=A), EINVAL)]
    + [(dict({**NO_NORM, k: A}), EINVAL) for k in ("beta", "z", "rstd", "q", "e")],
    "oba_residual_norm_backward": [
        (dict(alpha=-1e39), EINVAL),
        (dict(n=0), EINVAL), (dict(n=4097), EINVAL), (dict(rows=-1), EINVAL),
        (dict(rows=1 << 30), EINVAL), (dict(cols=0), EINVAL), (dict(cols=16385), EINVAL),
        (dict(dtype=3), EINVAL), (dict(g_dtype=-1), EINVAL), (dict(kind=2), EINVAL),
        (dict(alpha=NAN), EINVAL), (dict(rate=2.0), EINVAL), (dict(lddz=8), EINVAL),
        (dict(lddr=39), EINVAL), (dict(lddx=32), EINVAL), (dict(lddb=36), EINVAL),
        (dict(ldg=39), EINVAL), (dict(dz=None), EINVAL), (dict(dz=A + 8), EALIGN),
        (dict(q=None), EINVAL), (dict(e=None), EINVAL), (dict(q=A + 8), EALIGN),
        (dict(rstd=None), EINVAL), (dict(gamma=None), EINVAL), (dict(gamma=A + 2), EALIGN),
        (dict(dr=A + 4), EALIGN), (dict(dx=None), EINVAL), (dict(dx=A + 8), EALIGN),
        (dict(qb=None), EINVAL), (dict(eb=None), EINVAL), (dict(qb=None, eb=None), EINVAL),
        (dict(qb=A + 8), EALIGN), (dict(rstd_b=None), EINVAL), (dict(gamma_b=None), EINVAL),
        (dict(beta_b=A + 2), EALIGN), (dict(gate=None), EINVAL), (dict(gate=A + 1), EALIGN),
        (dict(rng=None), EINVAL), (dict(db=A + 8), EALIGN), (dict(dgamma=A + 1), EALIGN),
        (dict(dgate=A + 1), EALIGN), (dict(ws=None), EINVAL), (dict(ws=A + 8), EALIGN),
        (dict(ws_bytes=8), EWORKSPACE), (dict(NO_DZ, dr=None), EINVAL),
        (dict({**NO_DZ, "dz": A}), EINVAL), (dict({**NO_DZ, "rstd": A}), EINVAL),
        (dict({**NO_DZ, "dgamma": A}), EINVAL), (dict({**NO_DZ, "dbeta": A}), EINVAL),
        (dict(gamma_b=None, beta_b=None, rstd_b=None), EINVAL)],
    "oba_gated_linear": [
        (dict(rows=-1), EINVAL), (dict(n_in=0), EINVAL), (dict(hidden=0), EINVAL),
        (dict(hidden=-8), EINVAL), (dict(hidden=(1 << 19) + 8, ldy=1 << 20), EINVAL),
        (dict(hidden=1 << 62, ldy=1 << 20), EINVAL), (dict(dtype=F32), EINVAL),
        (dict(gate=6), EINVAL), (dict(gate=-1), EINVAL), (dict(ldx=2040), EINVAL),
        (dict(ldw=2049), EINVAL), (dict(ldy=56), EINVAL), (dict(x=None), EINVAL),
        (dict(w=None), EINVAL), (dict(y=None), EINVAL), (dict(x=A + 2), EALIGN),
        (dict(w=A + 8), EALIGN), (dict(y=A + 4), EALIGN), (dict(bias=A + 2), EALIGN),
        (dict(qp=None), EINVAL), (dict(ep=None), EINVAL), (dict(qu=None), EINVAL),
        (dict(eu=None), EINVAL), (dict(qp=None, ep=None), EINVAL),
        (dict(qu=None, eu=None), EINVAL), (dict(qu=A + 8), EALIGN), (dict(q=None), EINVAL),
        (dict(e=None), EINVAL), (dict(ws=None), EINVAL), (dict(ws=A + 4), EALIGN),
        (dict(ws_bytes=0), EWORKSPACE)],
    "oba_gated_hidden_grad": [
        (dict(rows=-1), EINVAL), (dict(n_out=0), EINVAL), (dict(hidden=0), EINVAL),
        (dict(hidden=(1 << 19) + 8, ldw=1 << 20, lddpu=1 << 21), EINVAL), (dict(dtype=F32), EINVAL),
        (dict(gate=6), EINVAL), (dict(lddy=2040), EINVAL), (dict(ldw=56), EINVAL),
        (dict(lddpu=120), EINVAL), (dict(dy=None), EINVAL), (dict(w=None), EINVAL),
        (dict(dpu=None), EINVAL), (dict(dy=A + 8), EALIGN), (dict(w=A + 2), EALIGN),
        (dict(dpu=A + 8), EALIGN), (dict(qp=None), EINVAL), (dict(ep=None), EINVAL),
        (dict(qu=None), EINVAL), (dict(eu=None), EINVAL), (dict(qp=A + 8), EALIGN),
        (dict(ws=None), EINVAL), (dict(ws_bytes=64), EWORKSPACE)],
}


@no_gpu
@pytest.mark.parametrize("name,change,expect", [(n, c, x) for n, cs in CASES.items()
                                                for c, x in cs])
def test_refused(name, change, expect):
    assert call(name, BASES[name], **change) == expect, change


@no_gpu
@pytest.mark.parametrize("name", list(BASES))
def test_good_arguments_reach_the_launch(name):
    """Where there is no GPU it fails; what is allowed to be absent may be."""
    base = BASES[name]
    assert call(name, base) == EHIP
    absent = {"oba_dropout": [dict(add=None), dict(rate=0.0, rng=None), dict(rate=1.0 - 2.0 ** -16)],
              "oba_residual_norm": [NO_BRANCH, NO_NORM, dict(r=None), dict(gate=None),
                                    dict(beta=None, beta_b=None), dict(q=None, e=None),
                                    dict(qb=None, eb=None), dict(NO_BRANCH, **NO_NORM),
                                    dict(rate=1e-9, rng=None)],
              "oba_residual_norm_backward": [
                  NO_DZ, dict(dr=None), dict(db=None), dict(gate=None, dgate=None),
                  dict(dbeta=None, dbeta_b=None, beta_b=None),
                  dict(dgamma=None, dbeta=None, dgamma_b=None, dbeta_b=None, dgate=None, ws=None,
                       ws_bytes=0, ldg=0)],
              "oba_gated_linear": [dict(bias=None), dict(q=None, e=None),
                                   dict(qp=None, ep=None, qu=None, eu=None)],
              "oba_gated_hidden_grad": [dict(gate=0)]}[name]
    for change in absent:
        assert call(name, base, **change) == EHIP, change


@no_gpu
@pytest.mark.parametrize("name", ["oba_dropout", "oba_residual_norm", "oba_gated_linear",
                                  "oba_gated_hidden_grad"])
def test_no_rows_need_no_memory(name):
    none = {k: None for k, v in BASES[name].items() if v == A}
    assert call(name, BASES[name], rows=0, **none) == 0


@no_gpu
@pytest.mark.parametrize("rows,hidden", [(1 << 30, 1 << 11), (1 << 24, 1 << 17)])
def test_sizes_that_one_launch_cannot_walk(rows, hidden):
    assert call("oba_gated_linear", GATED, rows=rows, n_in=8, ldx=8, ldw=8, hidden=hidden,
                ldy=hidden) == EINVAL
    assert call("oba_gated_hidden_grad", GRAD, rows=rows, n_out=8, lddy=8, hidden=hidden,
                ldw=hidden, lddpu=2 * hidden) == EINVAL


def test_workspace_sizes():
    L = oba.lib()
    assert L.oba_gated_linear_workspace_bytes(100, 2048, 64) > 0
    assert L.oba_gated_linear_workspace_bytes(16384, 1024, 4096) == 0
    assert L.oba_gated_linear_workspace_bytes(0, 64, 64) == 0
    assert L.oba_gated_linear_workspace_bytes(10, 64, 1 << 20) == 0
    assert L.oba_gated_hidden_grad_workspace_bytes(100, 64, 2048) > 0
    assert L.oba_gated_hidden_grad_workspace_bytes(16384, 4096, 1024) == 0
    assert L.oba_gated_hidden_grad_workspace_bytes(-1, 64, 64) == 0
    assert L.oba_residual_norm_backward_workspace_bytes(2, 4, 40) >= 2 * 4 * 40 * 4
    assert L.oba_residual_norm_backward_workspace_bytes(2, 4, 1 << 20) == 0


def test_binding_refuses_host_tensors_and_unknown_kinds(monkeypatch):
    import torch

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, v = torch.zeros(4, 40), torch.zeros(4)
    with pytest.raises(TypeError):
        oba.dropout(x, x, None, 0.0)
    with pytest.raises(TypeError):
        oba.residual_norm(x, 1e-5, r=x)
    with pytest.raises(TypeError):
        oba.residual_norm_backward(1, x, x, None, dr=x)
    with pytest.raises(TypeError):
        oba.gated_linear(x, x, x, None)
    with pytest.raises(TypeError):
        oba.gated_hidden_grad(x, x, None, None, None, None, x, None)
    c = oba._Call()
    with pytest.raises(TypeError):
        c.rng(v)
    assert set(oba.NORMS) == {"layer", "rms"}
    assert set(oba.GATES) == {"none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"}
