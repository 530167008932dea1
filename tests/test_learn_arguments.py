"""Arguments that the learned parts' Python calls refuse (no GPU needed)."""
from __future__ import annotations

import pytest
import torch


@pytest.mark.parametrize("coeffs", [(1.5, -0.5), (1.5,), (1.0, 0.0, 0.0, 0.0), ()])
def test_orthogonalize_wants_three_coefficients(monkeypatch, coeffs):
    """Two of them are not a polynomial whose third is zero."""
    from splat_rendering_gb300 import pulsar as pl
    ops = object.__new__(pl.Learner)
    ops.handle, ops.device, ops._torch, ops._dev = 0, 0, torch, "cpu"
    monkeypatch.setattr(pl.Learner, "_tensor", lambda self, t, *a: t.data_ptr())
    monkeypatch.setattr(pl.Learner, "_stream", lambda self, s: 0)

    class Library:
        @staticmethod
        def pulsar_orthogonalize(*args):
            raise AssertionError("the call reached the library")

    ops._lib = Library
    with pytest.raises(ValueError, match="coeffs"):
        ops.orthogonalize(torch.ones(2, 3), coeffs=coeffs)
