"""The learned parts together, as the training example uses them."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "learn_codebook", os.path.join(ROOT, "examples", "learn_codebook.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_loss_falls():
    losses = _example().train(steps=30, spheres=3000, rows=64, size=96)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.5 * losses[0], (losses[0], losses[-1])


def test_step_gradient_is_the_loss_derivative():
    """Central differences of the whole step's loss along its own codebook and
    norm gradients.  The network rounds to 16 bits, so the loss is a staircase
    at the scale of its rounding (2^-8 of an activation, averaged over the
    image's pixels); a step of 1e-2 of the parameters' scale stands a hundred
    times above that, and 5 percent covers it and the curvature."""
    ex = _example()
    model = ex.Model(3000, 64, 96, seed=3)
    target = model.forward() * 0.5
    n = target.numel()

    def loss():
        return float(((model.forward() - target) ** 2).double().mean())

    grads = model.backward((model.forward() - target) * (2.0 / n))
    for name, g in zip(("codebook", "gamma", "beta"), grads):
        p = getattr(model, name)
        d = g / g.norm() * p.numel() ** 0.5
        h = 1e-2
        setattr(model, name, p + h * d)
        up = loss()
        setattr(model, name, p - h * d)
        down = loss()
        setattr(model, name, p)
        want = float((g * d).sum())
        assert abs((up - down) / (2 * h) - want) <= 0.05 * abs(want), (name, (up - down) / (2 * h), want)
    model.close()
