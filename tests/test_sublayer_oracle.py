"""The plain forms that the sub-layer's operators are tested against, checked on
the CPU: the generator against its published known answers, the norms' and the
gates' gradients against differences."""
import numpy as np
import pytest
import torch

from sublayer_common import GATES, factor, gate64, norm_rows64, philox, through64


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_generator_has_its_published_answers(counter, key, words):
    assert tuple(int(v) for v in philox(counter, key)) == words


def test_share_of_dropped_elements():
    """Binomial: within five standard deviations of the rate as rounded."""
    for rate in (0.1, 0.5, 0.9):
        n = 400 * 1000
        p = round(rate * 65536) / 65536
        f = factor(400, 1000, rate, seed=1234567890123, step=7, site=3)
        assert abs((f == 0).sum() - n * p) <= 5 * (n * p * (1 - p)) ** 0.5
        assert np.all((f == 0) | (f == 1 / (1 - p)))
    assert np.all(factor(3, 5, 0.0, 1, 2, 3) == 1.0)


@pytest.mark.parametrize("kind", GATES)
def test_gate_derivatives(kind):
    p = torch.linspace(-9, 9, 360, dtype=torch.float64) + 0.013  # not at relu's corner
    h = 1e-6
    slope = (gate64(p + h, kind)[0] - gate64(p - h, kind)[0]) / (2 * h)
    # h^2 times a third derivative below 2, and two values below 10 that are off by
    # up to 4 units of 2^-53 (an exponential, a quotient, a product), over 2 h:
    # 8 * 10 * 1.2e-16 / 2e-6
    assert bool(((gate64(p, kind)[1] - slope).abs() <= 2 * h * h + 4.8e-9).all())


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient(kind):
    g = torch.Generator().manual_seed(1)
    x, v, w = (torch.randn((4, 33), generator=g, dtype=torch.float64) for _ in range(3))
    h = 1e-6
    up, dn = norm_rows64(x + h * v, 1e-5, kind)[0], norm_rows64(x - h * v, 1e-5, kind)[0]
    hx, rs = norm_rows64(x, 1e-5, kind)
    slope = float((through64(w, hx, rs, kind) * v).sum())
    assert abs(float(((up - dn) / (2 * h) * w).sum()) - slope) <= 1e-7 * float((w * v).abs().sum())
