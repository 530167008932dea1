"""Orthogonalisation of tensors that begin at any element of their memory, as
the slices of a flat parameter vector do."""
from __future__ import annotations

import pytest
import torch

import learn_reference as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
COEFFS = tuple(float(torch.tensor(v, dtype=torch.float32)) for v in (3.4445, -4.775, 2.0315))
EPS = float(torch.tensor(1e-7, dtype=torch.float32))


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=1 << 26)
    yield o
    assert o.status() == 0
    o.close()


def _at(offset, shape, dtype):
    """A tensor that begins `offset` elements into its memory, between guards."""
    n = 1
    for d in shape:
        n *= d
    flat = torch.full((n + offset + 16,), 77.0, device="cuda", dtype=dtype)
    return flat, flat[offset:offset + n].view(shape)


# on chip, alone and by a cluster; by separate products; tall and odd ones
SHAPES = [(64, 64), (3, 16, 64), (8, 1000), (128, 512), (64, 19), (40, 24), (300, 400), (400, 300),
          (200, 333)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offsets", [(0, 1), (1, 0), (1, 1), (0, 2), (3, 2)],
                         ids=lambda o: f"grad{o[0]}-out{o[1]}")
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_any_element_alignment(ops, shape, offsets, dtype):
    T = TYPES[dtype]
    g = torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).to(T)
    _, grad = _at(offsets[0], shape, T)
    grad.copy_(g)
    flat, out = _at(offsets[1], shape, T)
    assert ops.orthogonalize(grad, out=out) is out
    want, bound = ref.orthogonalize(g, 5, COEFFS, EPS)
    got = out.cpu().double()
    assert ((got - want).flatten(-2).norm(dim=-1) <= bound).all()
    # the aligned form sums the norm in another order; in 16 bits both are rounded once more, and
    # each is within 2^-9 of its norm of the exact result besides
    whole = ops.orthogonalize(g.cuda()).cpu().double()
    assert (got - whole).norm() <= (1e-5 if dtype == "f32" else 2.0 ** -7) * whole.norm()
    assert flat[:offsets[1]].eq(77).all() and flat[offsets[1] + out.numel():].eq(77).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_in_a_flat_vector(ops, dtype):
    """Two matrices side by side in one vector, the second off every boundary."""
    T = TYPES[dtype]
    gen = torch.Generator().manual_seed(5)
    flat = torch.randn(3 * 7 + 64 * 64, generator=gen).to(T).cuda()
    first, second = flat[:21].view(3, 7), flat[21:].view(64, 64)
    want = ops.orthogonalize(first.clone()), ops.orthogonalize(second.clone())
    for m, w in zip((first, second), want):
        ops.orthogonalize(m, out=m)
        assert (m.double() - w.double()).norm() <= (1e-5 if dtype == "f32" else 2.0 ** -7) * w.double().norm()
