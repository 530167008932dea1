"""Every form of the orthogonalisation's products, and every shape in 16 bits,
against the definition in 64 bits with criteria that an empty result fails.

16 bits: the arithmetic may add as much error as the rounding of the result
has by itself, sqrt(2) of it together; 2^-13 of the result on top stands for
matrices of so few elements that one value near the middle of two neighbours,
rounded to the other one, is much of their error.
32 bits: no more than twice as far off as plain 32-bit products."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
COEFFS = tuple(float(torch.tensor(v, dtype=torch.float32)) for v in (3.4445, -4.775, 2.0315))
EPS = float(torch.tensor(1e-7, dtype=torch.float32))


def _plain(x):
    a, b, c = COEFFS
    if tall := x.shape[-2] > x.shape[-1]:
        x = x.mT
    x = x / (x.pow(2).sum((-1, -2), keepdim=True).sqrt() + EPS)
    for _ in range(5):
        A = x @ x.mT
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.mT if tall else x


def _norm(x):
    return x.flatten(-2).norm(dim=-1)


def _gradient(B, m, n, seed):
    """Some strong directions above a noise floor."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    k = max(1, min(m, n) // 8)
    return 1e-3 * (r(B, m, k) @ r(B, k, n) / k ** 0.5 + 0.5 * r(B, m, n))


def _check(g):
    from splat_rendering_gb300 import pulsar as pl
    ops = pl.Learner(workspace_bytes=pl.orthogonalize_workspace(*g.shape, g.dtype))
    got = ops.orthogonalize(g)
    assert ops.status() == 0
    ops.close()
    for i in range(0, g.shape[0], 16):
        part = slice(i, i + 16)
        want = _plain(g[part].double())
        err = _norm(got[part].double() - want)
        if g.dtype == torch.bfloat16:
            bound = 2 ** 0.5 * _norm(want.float().bfloat16().double() - want) + 2.0 ** -13 * _norm(want)
        else:
            bound = 2 * _norm(_plain(g[part]).double() - want)
        assert (err <= bound).all(), (i, float((err / bound).max()))


SMALL = [
    (1, 1, 1), (3, 1, 7), (2, 9, 1), (8, 64, 64), (4, 64, 19), (5, 3, 64), (1, 16, 700),
    (1, 2000, 16), (2, 65, 64), (1, 127, 129), (1, 128, 128), (1, 200, 100), (2, 150, 300),
    (1, 513, 257), (1, 300, 1025), (33, 20, 31), (1, 128, 3000), (1, 640, 512), (1, 512, 768),
    (1, 1301, 1154), (1, 10, 3000), (2, 100, 900), (1, 5000, 30), (3, 128, 1024), (1, 7, 2100),
    (40, 50, 600), (1, 128, 2000), (1, 2, 40000),
]


@pytest.mark.parametrize("case", SMALL, ids=lambda c: "-".join(map(str, c)))
def test_sixteen_bits_at_every_shape(case):
    B, m, n = case
    _check(_gradient(B, m, n, B * 31 + m * 7 + n).bfloat16())


# the symmetric products of 128 x 256 shared by two CTAs and the last product of 256 columns; the
# latter with odd remainders; symmetric products of one CTA each, several tiles a CTA
FORMS = [(1, 2048, 4096), (1, 4000, 1900), (30, 200, 300), (1, 2100, 2300), (100, 200, 300),
         (20, 500, 700), (3, 1280, 1100)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", FORMS, ids=lambda c: "-".join(map(str, c)))
def test_forms_of_the_products(case, dtype):
    _check(_gradient(*case, sum(case)).to(dtype))


def test_products_of_more_elements_than_31_bits():
    """Every offset of the products is 64 bits wide: matrices that repeat give
    results that repeat, the first of them checked."""
    from splat_rendering_gb300 import pulsar as pl
    B, m, n = 10_000, 200, 1100
    assert B * m * n > 1 << 31
    need = pl.orthogonalize_workspace(B, m, n, torch.bfloat16)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need + (16 << 30):
        pytest.skip("not enough device memory")
    one = _gradient(1, m, n, 7).bfloat16()
    grad = one.repeat(B, 1, 1)
    ops = pl.Learner(workspace_bytes=need)
    out = ops.orthogonalize(grad, out=grad)
    want = _plain(one[0].double())
    err = (out[0].double() - want).norm()
    assert err <= 2 ** 0.5 * (want.float().bfloat16().double() - want).norm() + 2.0 ** -13 * want.norm()
    assert torch.equal(out.amax(0), out[0]) and torch.equal(out.amin(0), out[0])
    assert ops.status() == 0
    ops.close()
