"""Newton-Schulz orthogonalisation against its definition in 64 bits."""
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
    o = pl.Learner(workspace_bytes=1 << 29)
    yield o
    assert o.status() == 0
    o.close()


def _check(got, grad, steps=5, coeffs=COEFFS):
    want, bound = ref.orthogonalize(grad, steps, coeffs, EPS)
    err = (got.cpu().double() - want).flatten(-2).norm(dim=-1)
    assert got.dtype == grad.dtype and got.shape == grad.shape
    assert (err <= bound).all(), (float((err / bound.clamp(min=1e-300)).max()))
    return err / want.flatten(-2).norm(dim=-1).clamp(min=1e-300)


CASES = [
    # batch, m, n
    (1, 1, 1), (3, 1, 7), (2, 9, 1), (8, 64, 64), (4, 64, 19), (5, 3, 64), (1, 16, 700),
    (1, 2000, 16), (2, 65, 64), (1, 127, 129), (1, 128, 128), (1, 200, 100), (2, 150, 300),
    (1, 513, 257), (1, 300, 1025), (33, 20, 31), (1, 128, 3000), (1, 640, 512), (1, 512, 768),
    (1, 1301, 1154), (1, 10, 3000), (2, 100, 900), (1, 5000, 30), (3, 128, 1024), (1, 7, 2100),
    (40, 50, 600), (1, 128, 2000), (1, 2, 40000),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_orthogonalize(ops, case, dtype):
    B, m, n = case
    gen = torch.Generator().manual_seed(B * 31 + m * 7 + n)
    k = max(1, min(m, n) // 8)
    g = torch.randn(B, m, k, generator=gen) @ torch.randn(B, k, n, generator=gen) / k ** 0.5
    g = (1e-3 * (g + 0.5 * torch.randn(B, m, n, generator=gen))).to(TYPES[dtype])
    _check(ops.orthogonalize(g.cuda()), g)


@pytest.mark.parametrize("shape", [(1, 35, 1330), (2, 4, 318), (1, 436, 3), (8, 5, 6), (16, 2, 10),
                                   (2, 39, 513), (8, 64, 64), (1, 128, 512), (1, 100, 4000),
                                   (2, 300, 400), (1, 4096, 350), (1, 512, 8192)],
                         ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("same", [False, True], ids=["normal", "orthogonal"])
def test_sixteen_bits_lose_no_more_than_their_result(ops, shape, same):
    """In 16 bits the arithmetic may add as much error as the rounding of the
    result has by itself: sqrt(2) of it together.  Roundings that are alike in
    every row (nearly orthogonal rows have nearly equal diagonals) would not
    average out and break this."""
    for seed in range(3):
        gen = torch.Generator().manual_seed(seed)
        g = torch.randn(*shape, generator=gen)
        if same:
            g = torch.linalg.svd(g.double(), full_matrices=False)
            g = (g.U @ g.Vh).float()
        g = g.bfloat16()
        want, _ = ref.orthogonalize(g, 5, COEFFS, EPS)
        err = (ops.orthogonalize(g.cuda()).cpu().double() - want).norm()
        own = (want.float().bfloat16().double() - want).norm()
        assert err <= 2 ** 0.5 * own, float(err / own)


@pytest.mark.parametrize("shape", [(4, 3, 190), (8, 5, 51), (13, 8, 184), (8, 64, 64),
                                   (1, 35, 1330), (1, 128, 2000), (1, 200, 300), (1, 1500, 509),
                                   (1, 683, 2967), (1, 1024, 1024)],
                         ids=lambda c: "-".join(map(str, c)))
def test_thirty_two_bits_are_those_of_plain_products(ops, shape):
    """In 32 bits the result is as near as that of plain 32-bit products: no
    more than twice as far off, over four matrices."""
    ours = plain = 0.0
    for seed in range(4):
        g = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()
        want, x = g.double(), g
        a, b, c = COEFFS

        def steps(x):
            if tall := x.shape[-2] > x.shape[-1]:
                x = x.mT
            x = x / (x.pow(2).sum((-1, -2), keepdim=True).sqrt() + EPS)
            for _ in range(5):
                A = x @ x.mT
                x = a * x + (b * A + c * (A @ A)) @ x
            return x.mT if tall else x

        want, x = steps(want), steps(x)
        ours += float((ops.orthogonalize(g).double() - want).norm() / want.norm())
        plain += float((x.double() - want).norm() / want.norm())
    assert ours <= 2 * plain, ours / plain


def test_singular_values_go_to_one(ops):
    """The polynomial takes singular values of a well-conditioned matrix into
    [0.65, 1.25] and keeps the singular vectors: U^T out V is diagonal."""
    gen = torch.Generator().manual_seed(2)
    u, _ = torch.linalg.qr(torch.randn(96, 96, generator=gen).double())
    v, _ = torch.linalg.qr(torch.randn(160, 96, generator=gen).double())
    s = torch.logspace(0, -1.5, 96, dtype=torch.float64)
    out = ops.orthogonalize(((u * s) @ v.mT).float().cuda()).cpu().double()
    core = u.mT @ out @ v
    d = core.diagonal()
    assert (d > 0.65).all() and (d < 1.25).all()
    assert (core - torch.diag(d)).abs().max() < 1e-3


@pytest.mark.parametrize("steps", [0, 1, 2, 9])
def test_steps_and_other_coefficients(ops, steps):
    gen = torch.Generator().manual_seed(steps)
    for shape in ((40, 70), (260, 140)):
        g = torch.randn(*shape, generator=gen)
        _check(ops.orthogonalize(g.cuda(), steps=steps, coeffs=(1.5, -0.5, 0.0)), g, steps,
               (1.5, -0.5, 0.0))


def test_zero_matrix_low_rank_and_scales(ops):
    gen = torch.Generator().manual_seed(17)
    for m, n in ((50, 60), (300, 200)):
        assert ops.orthogonalize(torch.zeros(2, m, n, device="cuda")).eq(0).all()
        one = torch.outer(torch.randn(m, generator=gen), torch.randn(n, generator=gen))
        for scale in (1.0, 1e-3, 1e15, 1e25):
            _check(ops.orthogonalize((one * scale).cuda()), one * scale)
        # a matrix of the batch does not see its neighbours
        g = torch.randn(3, m, n, generator=gen)
        g[1] = float("nan")
        out = ops.orthogonalize(g.cuda()).cpu()
        assert out[1].isnan().all()
        alone = ops.orthogonalize(g[2].contiguous().cuda()).cpu()
        assert out[0].isfinite().all() and torch.equal(out[2], alone)


def test_transpose_and_in_place(ops):
    gen = torch.Generator().manual_seed(19)
    for m, n in ((64, 19), (300, 170)):
        g = torch.randn(m, n, generator=gen).cuda()
        a = ops.orthogonalize(g)
        b = ops.orthogonalize(g.t().contiguous())
        # the same products up to their order
        assert (a - b.t()).norm() <= 1e-5 * a.norm()
        z = g.clone()
        ops.orthogonalize(z, out=z)
        assert torch.equal(z, a)


def test_same_bits_every_time_and_on_another_stream(ops):
    gen = torch.Generator().manual_seed(23)
    for shape in ((8, 64, 64), (400, 300)):
        g = torch.randn(*shape, generator=gen).cuda()
        want = ops.orthogonalize(g)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = ops.orthogonalize(g)
        s.synchronize()
        assert torch.equal(got, want)


def test_nothing_to_do(ops):
    for shape in ((0, 4, 4), (3, 0, 4), (2, 4, 0)):
        assert ops.orthogonalize(torch.empty(shape, device="cuda")).shape == shape


def test_refusals(ops):
    from splat_rendering_gb300 import pulsar as pl
    g = torch.zeros(8, 4, device="cuda")
    with pytest.raises(ValueError, match="not contiguous"):
        ops.orthogonalize(g.t())
    with pytest.raises(ValueError, match="shape"):
        ops.orthogonalize(g[0])
    with pytest.raises(TypeError):
        ops.orthogonalize(g.half())
    for kw in (dict(steps=-1), dict(eps=-1.0), dict(coeffs=(1.0, float("nan"), 0.0))):
        with pytest.raises(pl.PulsarError):
            ops.orthogonalize(g, **kw)
    small = pl.Learner(workspace_bytes=0)
    with pytest.raises(pl.PulsarError, match="workspace"):
        small.orthogonalize(torch.zeros(500, 500, device="cuda"))
    small.close()
