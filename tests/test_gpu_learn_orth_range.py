"""Orthogonalisation of matrices whose norm, or its square, is outside float32's
range, with and without an eps."""
from __future__ import annotations

import pytest
import torch

import learn_reference as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
COEFFS = tuple(float(torch.tensor(v, dtype=torch.float32)) for v in (3.4445, -4.775, 2.0315))
SHAPES = [(3, 40, 60), (16, 700), (2, 300, 200), (130, 140)]   # on chip, and by products
_ids = dict(ids=lambda c: "-".join(map(str, c)))


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=1 << 27)
    yield o
    assert o.status() == 0
    o.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, **_ids)
def test_a_power_of_two_changes_no_bit(ops, shape, dtype):
    """With eps = 0 the result does not depend on the matrix's scale: a power
    of two goes through every operation exactly, whatever the norm (its square
    below float32's range, or itself above it)."""
    g = torch.randn(*shape, generator=torch.Generator().manual_seed(1)).clamp(-4, 4)
    g = torch.where(g.abs() < 2.0 ** -4, 0.5, g).to(TYPES[dtype]).cuda()
    want = ops.orthogonalize(g, eps=0.0)
    assert want.isfinite().all() and want.ne(0).any()
    for k in (-120, -100, -80, -60, -41, -40, -39, -20, 20, 50, 60, 64, 100, 120, 125):
        got = ops.orthogonalize(g * 2.0 ** k, eps=0.0)
        assert torch.equal(got, want), k


@pytest.mark.parametrize("shape", SHAPES, **_ids)
def test_zero_stays_zero_without_eps(ops, shape):
    for T in TYPES.values():
        for steps in (0, 5):
            out = ops.orthogonalize(torch.zeros(shape, device="cuda", dtype=T), steps=steps, eps=0.0)
            assert out.eq(0).all()


@pytest.mark.parametrize("shape", SHAPES, **_ids)
def test_no_steps_at_the_ends_of_the_range(ops, shape):
    """No step: G / (|G| + eps), four roundings and the norm's sum of squares,
    whose terms are added in runs of at most 2^10 per thread."""
    for scale in (2.0 ** -130, 1e-30, 1e-22, 1e22, 2.0 ** 124):
        g = (torch.randn(*shape, generator=torch.Generator().manual_seed(3)).clamp(-4, 4) * scale)
        want, _ = ref.orthogonalize(g, 0, COEFFS, 0.0)
        got = ops.orthogonalize(g.cuda(), steps=0, eps=0.0).cpu().double()
        assert (got - want).norm() <= 2.0 ** -13 * want.norm(), scale
