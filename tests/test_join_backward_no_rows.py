"""The join's backward pass without rows still reads the parameters for their gradients'
zeros: what it reads is checked."""
import pytest

from test_sublayer_refusals import A, BACK, EALIGN, EHIP, call, no_gpu

NAME = "oba_residual_norm_backward"


@no_gpu
@pytest.mark.parametrize("name", ["gamma_b", "beta_b", "gate"])
def test_parameters_not_aligned(name):
    assert call(NAME, BACK, rows=0, **{name: A + 2}) == EALIGN
    assert call(NAME, BACK, rows=0, **{name: A + 4}) == EHIP


@no_gpu
def test_nothing_asked_for():
    none = {k: None for k, v in BACK.items() if v == A}
    assert call(NAME, BACK, rows=0, **none) == 0
