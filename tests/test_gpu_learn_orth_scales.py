"""Orthogonalisation of matrices far below eps and with coefficients far
from the usual, against its definition in 64 bits."""
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


def _f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, **_ids)
def test_matrices_far_below_eps(ops, shape, dtype):
    """|G| far below eps: X_0 is G / eps and stays small, so that a step is a X
    and the reference's bound is a few roundings of the products."""
    for scale in (1e-9, 1e-12, 1e-16, 1e-18, 1e-25):
        gen = torch.Generator().manual_seed(2)
        g = (torch.randn(*shape, generator=gen) * scale).to(TYPES[dtype])
        for eps in (1e-7, 0.5):
            got = ops.orthogonalize(g.cuda(), eps=eps).cpu().double()
            want, bound = ref.orthogonalize(g, 5, COEFFS, _f32(eps))
            err = (got - want).flatten(-2).norm(dim=-1)
            assert scale == 1e-9 or (bound <= 0.01 * want.flatten(-2).norm(dim=-1)).all()
            assert (err <= bound).all(), (scale, eps, float((err / bound).max()))


@pytest.mark.parametrize("case", [(1, (1000.0, 0.0, 0.0)), (3, (100.0, 0.0, 0.0)), (1, (3e5, 0.0, 0.0)),
                                  (5, (0.01, 0.0, 0.0)), (3, (2.0, 5.0, 5.0)), (2, (-90.0, 20.0, -3.0)),
                                  (4, (0.0, 0.0, 0.0)), (1, (0.0, 5000.0, 0.0))],
                         ids=lambda c: f"{c[0]}x{c[1]}")
@pytest.mark.parametrize("shape", SHAPES, **_ids)
def test_coefficients_far_from_the_usual(ops, shape, case):
    """Polynomials that grow or shrink the iterates by orders of magnitude."""
    steps, coeffs = case
    coeffs = tuple(_f32(v) for v in coeffs)
    for T in TYPES.values():
        g = torch.randn(*shape, generator=torch.Generator().manual_seed(4)).to(T)
        want, bound = ref.orthogonalize(g, steps, coeffs, _f32(1e-7))
        got = ops.orthogonalize(g.cuda(), steps=steps, coeffs=coeffs).cpu().double()
        err = (got - want).flatten(-2).norm(dim=-1)
        assert (err <= bound).all(), (T, float((err / bound.clamp(min=1e-300)).max()))


def test_coefficients_that_leave_the_range_are_refused(ops):
    from splat_rendering_gb300 import pulsar as pl
    g = torch.randn(20, 30, device="cuda")
    for steps, coeffs in ((2, (1e20, 0.0, 0.0)), (1, (1e30, -1e30, 0.0)), (12, (50.0, 3.0, 3.0)),
                          (100, (1.0, 1.0, 1.0))):
        with pytest.raises(pl.PulsarError):
            ops.orthogonalize(g, steps=steps, coeffs=coeffs)
    ops.orthogonalize(g, steps=100, coeffs=(1.5, -0.5, 0.0))


@pytest.mark.parametrize("scale", [1.0, 1e-9, 1e-14])
@pytest.mark.parametrize("steps", [60, 100])
def test_many_steps_end_at_the_polar_factor(ops, steps, scale):
    """(1.5, -0.5, 0) takes every singular value to 1, where its slope is zero:
    what is left is the last step's own rounding, (|a| + 3 |b|) 2^-20 |X|_F,
    and as much again for what the one before moved.  Matrices far below eps
    spend their first steps on growing (1.5^60 = 4e10)."""
    for shape in SHAPES:
        g = torch.randn(*shape, generator=torch.Generator().manual_seed(5)).double()
        u, _, vh = torch.linalg.svd(g, full_matrices=False)
        s = torch.linspace(1.0, 0.2, u.shape[-1], dtype=torch.float64)
        g = (scale * (u * s) @ vh).float()
        got = ops.orthogonalize(g.cuda(), steps=steps, coeffs=(1.5, -0.5, 0.0)).cpu().double()
        want = u @ vh   # (the polar factor; the rounding of g to 32 bits moves it by 2^-24 / 0.2)
        err = (got - want).flatten(-2).norm(dim=-1)
        assert (err <= 8 * 2.0 ** -20 * want.flatten(-2).norm(dim=-1)).all(), (shape, err)


@pytest.mark.parametrize("eps", [1.0, 3e4, 1e13, 1e20])
def test_a_large_eps(ops, eps):
    """X_0 is G / eps whatever the norm, whose square is below float32's range."""
    for shape in SHAPES:
        for scale in (1e-3, 1e-13, 1e-17):
            g = torch.randn(*shape, generator=torch.Generator().manual_seed(6)) * scale
            got = ops.orthogonalize(g.cuda(), eps=eps).cpu().double()
            want, bound = ref.orthogonalize(g, 5, COEFFS, _f32(eps))
            err = (got - want).flatten(-2).norm(dim=-1)
            # (below 2^-126 a result has the spacing of float32's subnormals)
            floor = 2.0 ** -150 * (shape[-1] * shape[-2]) ** 0.5
            assert (err <= bound + floor).all(), (shape, scale, float((err / bound).max()))
