"""A stream handed to a layer call belongs to the device that its tensors are
on: kernels launched on another device's stream would run there."""
from types import SimpleNamespace

import pytest

from communication_compressed_optimizer_02_amd import binding as oba


def test_a_stream_of_another_device_is_refused(monkeypatch):
    import torch

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    c = oba._Call()
    assert c.stream(SimpleNamespace(device_index=0, cuda_stream=77)) == 77
    with pytest.raises(ValueError, match="stream"):
        c.stream(SimpleNamespace(device_index=1, cuda_stream=77))
