"""Calls of the feed-forward sub-layer in an order that has nothing to read,
and instances that share their scratch."""
import sys

import pytest

from communication_compressed_optimizer_02_amd import FeedForward, synth
from communication_compressed_optimizer_02_amd import binding as oba
from layer_common import gen, rows, torch

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def test_backward_without_forward_is_refused():
    """Before the first forward() the kept tensors hold nothing."""
    t = torch()
    F = FeedForward(40, 72, 2, 3)
    L = oba.Layout(F.size, 2, synth.whole(F.size), synth.even_shards(F.size, 2))
    S = oba.State(L, "bf16")
    dy = t.ones((6, 40), device="cuda", dtype=t.bfloat16)
    S.g.fill_(7.0)
    with pytest.raises(RuntimeError):  # no parameters yet
        F.backward(dy, S.g)
    F.init(S.x)
    F.load(S.x)
    with pytest.raises(RuntimeError):
        F.backward(dy, S.g)
    t.cuda.synchronize()
    assert bool((S.g == 7.0).all()), "refused, but gradients were written"
    F.forward(dy)
    F.backward(dy, S.g)
    t.cuda.synchronize()
    assert bool(S.g[:, :F.size].isfinite().all())
    L.close()
