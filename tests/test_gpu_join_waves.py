"""Joins of every number of waves to a row, each with a last wave that the row does
not fill: forms of 8 columns a lane (512 columns to a wave) and of 16 (1024, above
8192 columns)."""
import pytest

import test_gpu_sublayer_calls as calls

pytestmark = pytest.mark.gpu

NARROW = [(w, 512 * w - 37) for w in range(1, 17)]
WIDE = [(w, 1024 * w - 37) for w in range(9, 17)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("w,c", NARROW + WIDE)
def test_rows_of_so_many_waves(w, c, dtype):
    assert -(-c // (512 if c <= 8192 else 1024)) == w
    calls.test_rows_of_every_number_of_waves(c, dtype)
