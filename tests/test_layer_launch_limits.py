"""Sizes that one launch cannot walk (HIP takes fewer than 2^32 threads) are
refused as sizes, not left to a failed launch.  Made-up addresses serve: the
refusals come before any HIP call."""
import ctypes
import os

import pytest

from communication_compressed_optimizer_02_amd import binding as oba

pytestmark = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                                reason="made-up addresses: not where a GPU could read them")
EINVAL, EHIP = -1, -5
F32, F16, BF16 = 0, 1, 2
AT = iter(range(1 << 46, 1 << 62, 1 << 46))  # addresses far apart: buffers do not overlap
X, Q, E, W, Y, R, WS, DB = (next(AT) for _ in range(8))


def call(name, *args):
    fn = getattr(oba.lib(), name)
    return fn(*[ctypes.c_void_p(v) if t is ctypes.c_void_p else v
                for v, t in zip(args, fn.argtypes)])


# 2^24 blocks are one too many: of 1024 pieces of 16 bytes, whole groups of 32
# columns to a row
@pytest.mark.parametrize("rows,cols,dtype", [
    (1 << 30, 33, F32), (1 << 30, 1 << 12, F32), (1 << 30, 97, BF16), (1 << 30, 1 << 12, F16),
    (1 << 24, 4096, F32), (1 << 24, 8161, BF16)])
def test_encode_and_decode(rows, cols, dtype):
    per_row = -(-cols // 32) * (8 if dtype == F32 else 4)
    blocks = -(-rows * per_row // 1024)
    ld = -(-cols // 8) * 8
    assert blocks >= 1 << 24
    assert call("oba_act8_encode", rows, cols, X, ld, dtype, Q, E, None) == EINVAL
    assert call("oba_act8_decode", rows, cols, Q, E, X, ld, dtype, None) == EINVAL


# results of 128 x 128 to a block
@pytest.mark.parametrize("rows,n_in,n_out", [
    (1 << 30, 8, 129), (1 << 30, 8, 1 << 12), (1 << 22, 8, 1 << 16)])
def test_products(rows, n_in, n_out):
    assert -(-rows // 128) * -(-n_out // 128) >= 1 << 24
    assert call("oba_linear", rows, n_in, n_out, X, n_in, W, n_in, BF16, None, 0, None, 0, Y, n_out
                + -n_out % 8, None, None, None, 0, None) == EINVAL
    assert call("oba_linear_input_grad", rows, n_out, n_in, X, n_in, W, n_out + -n_out % 8, F16, 0,
                None, None, None, 0, Y, n_out + -n_out % 8, None, 0, None) == EINVAL


@pytest.mark.parametrize("n,rows,n_in,n_out", [
    (4096, 1, 1 << 20, 1), (4096, 1, 1 << 19, 1), (4096, 2, 1 << 20, 1 << 12)])
def test_weight_gradients(n, rows, n_in, n_out):
    assert n * -(-n_in // 128) * -(-n_out // 128) >= 1 << 24
    for k in (rows, 0):
        assert call("oba_linear_weight_grad", n, k, n_in, n_out, X, n_out + -n_out % 8, BF16, Q, E,
                    W, DB, F32, n_in * n_out + n_out, WS, 1 << 40, None) == EINVAL


def test_the_largest_launch_is_not_refused():
    """One block less than too many: where there is no GPU, the launch fails."""
    r = (1 << 24) - 1
    assert call("oba_act8_encode", r, 8161, X, 8168, BF16, Q, E, None) == EHIP
    assert call("oba_act8_decode", r, 8161, Q, E, X, 8168, BF16, None) == EHIP
    assert call("oba_linear", 1 << 30, 8, 128, X, 8, W, 8, BF16, None, 0, None, 0, Y, 128, None,
                None, None, 0, None) == EHIP
