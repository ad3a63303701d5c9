"""The sequence operators together, as examples/sequence_block.py uses them: its gradients against
differences of its own loss, its training, and decoding against the whole sequence."""
from __future__ import annotations

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import sequence_block as E  # noqa: E402


def test_gradients_against_differences():
    """Central differences in float32 along one direction for each weight: the loss is a mean of some
    6000 terms of about 1, each off by some hundred roundings of 2^-24, most of which average out; its
    third derivatives are of order one. A step of 2^-6 of a direction of norm 1 keeps both under 2%
    of slopes that a random direction of the gradient itself has."""
    block = E.Block()
    x = E.tokens(torch.Generator().manual_seed(3), 2, 48, 64)
    want = torch.nn.functional.pad(x, (0, 0, 1, 0))[:, :-1]

    def loss():
        _, out, _ = block.forward(x)
        return float((out - want).double().square().mean())

    _, out, _ = block.forward(x)
    _, matrices, vectors = block.backward(torch.zeros_like(x), (out - want) * (2.0 / out.numel()))
    for name, grad in {**matrices, **vectors}.items():
        w = getattr(block, name)
        d = grad / grad.norm()
        kept = w.clone()
        step = 2.0 ** -6
        w.copy_(kept + step * d)
        up = loss()
        w.copy_(kept - step * d)
        down = loss()
        w.copy_(kept)
        slope, expected = (up - down) / (2 * step), float(grad.norm())
        assert abs(slope - expected) <= 0.02 * expected + 2.0 ** -24 * 100 / step, (name, slope, expected)


def test_training_and_decoding():
    block = E.Block()
    losses = E.train(block, 60, say=lambda *_: None)
    assert losses[-1] < 0.8 * losses[0], losses  # an untrained block's answers are unrelated
    # the same float32 sums in another order, through some ten operators
    assert E.decode(block) < 1e-4
