"""Orthogonalisation in 32 bits of a matrix so large that its typical entries
are 1e-4 of its norm: the lower halves of their pairs stay above half's
subnormals."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
COEFFS = tuple(float(torch.tensor(v, dtype=torch.float32)) for v in (3.4445, -4.775, 2.0315))
EPS = float(torch.tensor(1e-7, dtype=torch.float32))


def test_small_entries_keep_their_bits():
    """No more than twice as far off as plain 32-bit products."""
    from splat_rendering_gb300 import pulsar as pl
    m, n = 3000, 20_000
    g = torch.randn(m, n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    ops = pl.Learner(workspace_bytes=pl.orthogonalize_workspace(1, m, n, g.dtype))
    got = ops.orthogonalize(g)
    assert ops.status() == 0
    ops.close()

    def plain(x):
        a, b, c = COEFFS
        x = x / (x.pow(2).sum().sqrt() + EPS)
        for _ in range(5):
            A = x @ x.mT
            x = a * x + (b * A + c * (A @ A)) @ x
        return x

    want = plain(g.double())
    ours, theirs = (float((x.double() - want).norm() / want.norm()) for x in (got, plain(g)))
    assert ours <= 2 * theirs, (ours, theirs)
    print(ours, theirs)
