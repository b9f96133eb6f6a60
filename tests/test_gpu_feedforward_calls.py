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


def stack(share, n, r, width, hidden, dtype="bf16", layers=3):
    """(layers, state) of a stack whose parameters follow each other."""
    Fs, at = [], 0
    for k in range(layers):
        Fs.append(FeedForward(width, hidden, n, r, dtype, ("gelu", "relu", "none")[k % 3], at=at,
                              share=Fs[0] if share and Fs else None))
        at += Fs[-1].size
    L = oba.Layout(at, n, synth.whole(at), synth.even_shards(at, n))
    S = oba.State(L, "f32")
    g = gen(3)
    for F in Fs:
        F.init(S.x, g)
    return Fs, L, S


def test_a_stack_that_shares_scratch():
    """The same results as instances of their own, several steps in a row."""
    t = torch()
    say("[ff share] stack")
    n, r, width, hidden = 2, 45, 72, 200
    runs = []
    for share in (False, True):
        Fs, L, S = stack(share, n, r, width, hidden)
        g, out = gen(4), []
        for step in range(3):
            x, dy = rows(g, n * r, width, "bf16"), rows(g, n * r, width, "bf16", std=0.1)
            for F in Fs:
                F.load(S.x)
            for F in Fs:
                x = F.forward(x)
            out.append(x.clone())
            for F in reversed(Fs):
                dy = F.backward(dy, S.g)
            out += [dy.clone(), S.g.clone()]
            S.warmup(1e-3, 0.9, 0.999, 1e-8)
        t.cuda.synchronize()
        out.append(S.x.clone())
        assert all(bool(a.isfinite().all()) for a in out)
        runs.append(out)
        L.close()
    assert all(t.equal(a, b) for a, b in zip(*runs))


def test_memory_of_a_further_layer():
    """A layer that shares holds what its documentation says: 2 1/16 bytes per
    row and column of width and hidden, y and dx, rstd, the weights' copies."""
    t = torch()
    n, r, width, hidden = 4, 1024, 256, 1024
    first = FeedForward(width, hidden, n, r)
    t.cuda.synchronize()
    before = t.cuda.memory_allocated()
    second = FeedForward(width, hidden, n, r, share=first)
    held = t.cuda.memory_allocated() - before
    total = n * r
    stated = total * ((width + hidden) * 2 * 33 // 32 + 4 * width + 4) + 2 * 2 * width * hidden
    # each of 13 allocations in whole pieces of 512 bytes
    assert stated <= held <= stated + 13 * 512, (held, stated)
    # and as many 16-bit rows as a layer of its own holds beside that
    before = t.cuda.memory_allocated()
    third = FeedForward(width, hidden, n, r)
    held = t.cuda.memory_allocated() - before
    assert held >= stated + 4 * total * (width + hidden)
    del second, third


def test_sharing_needs_the_same_sizes():
    t = torch()
    F = FeedForward(40, 72, 2, 3)
    for args in ((48, 72, 2, 3), (40, 80, 2, 3), (40, 72, 3, 2), (40, 72, 2, 4),
                 (40, 72, 2, 3, "f16")):
        with pytest.raises(ValueError):
            FeedForward(*args, share=F)
    G = FeedForward(40, 72, 2, 3, act="relu", at=5, share=F)
    assert G.ws is F.ws and G.y.data_ptr() != F.y.data_ptr()
    t.cuda.synchronize()
