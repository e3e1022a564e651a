"""The example's training and decoding at small sizes."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx4_train_and_serve.py")
    spec = importlib.util.spec_from_file_location("mx4_train_and_serve", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_lowers_the_loss():
    losses = _example().train(tokens=1024, hidden=256, out=320, steps=40)
    assert all(a == a for a in losses) and losses[-1] < 0.1 * losses[0]


def test_decoding_steps_are_finite():
    us, y = _example().serve(experts=6, top_k=2, hidden=256, inner=96, tokens=5)
    assert us > 0 and torch.isfinite(y).all() and (y != 0).any()
