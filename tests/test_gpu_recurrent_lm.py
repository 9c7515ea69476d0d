"""The example model (examples/recurrent_lm.py): the layer operators and the delta rule together, in
training and one token at a time.

The two ways of scoring a token differ by the rounding of bf16 activations through two blocks (a few
2^-8 of hidden rows of unit mean square, logits of order one to ten): a mean difference of 0.05 is
several times that."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_lm.py")


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("recurrent_lm", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_trains_and_serves(lm):
    model = lm.Model()
    losses = lm.train(model, 60)
    assert all(l == l for l in losses) and losses[-1] < 0.8 * losses[0], (losses[0], losses[-1])
    test = lm.batch(3, 40, model.master["head"].shape[0], torch.Generator().manual_seed(5))
    whole, stepped = lm.score_both_ways(model, test)
    assert (whole - stepped).abs().mean().item() < 0.05
    made = lm.generate(model, test[:, :8], 4)
    assert made.shape == (3, 12) and torch.equal(made[:, :8], test[:, :8])


def test_gradients_reach_every_weight(lm):
    model = lm.Model(vocab=101, width=128, heads=2, hidden=200)
    model.cast()
    model.loss(lm.batch(2, 33, 101, torch.Generator().manual_seed(6))).backward()
    for name, w in model.master.items():
        assert w.grad is not None and torch.isfinite(w.grad).all() and w.grad.abs().sum() > 0, name
