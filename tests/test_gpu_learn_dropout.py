"""Dropout against its definition, its random numbers exactly."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=0)
    yield o
    assert o.status() == 0
    o.close()


def _check(got, x, p, seed, offset, residual):
    want, keep, bound = ref.dropout(x, p, seed, offset, residual)
    bad = ref.outside(got, want, bound)
    assert not bad.any(), int(bad.sum())
    return keep


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,p,seed,offset", [
    (1, 0.5, 0, 0), (3, 0.25, 1, 5), (4, 0.5, 2, 2 ** 32 - 1), (5, 0.9, 2 ** 64 - 1, 7),
    (31, 0.1, 2 ** 33 + 5, 0), (1000, 0.0, 3, 1), (4097, 0.333, 4, 2 ** 62), (100_003, 0.1, 5, 2 ** 32 - 100),
    (300_000, 0.7, 6, 2 ** 63 - 1), (77, 1.0 - 2.0 ** -32, 7, 0),
])
def test_dropout(ops, n, p, seed, offset, dtype, skip):
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=gen).to(TYPES[dtype])
    r = torch.randn(n, generator=gen).to(TYPES[dtype]) if skip else None
    y = ops.dropout(x.cuda(), p, seed, offset, residual=None if r is None else r.cuda())
    assert y.dtype == x.dtype
    _check(y, x, p, seed, offset, r)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_any_alignment_and_in_place(ops, dtype):
    T = TYPES[dtype]
    gen = torch.Generator().manual_seed(1)
    x, r = (torch.randn(5003, generator=gen).to(T) for _ in range(2))
    want = ops.dropout(x.cuda(), 0.4, 9, 11, residual=r.cuda())
    for shift in (1, 2, 3):
        off = lambda t: torch.cat([t[:1].expand(shift), t]).cuda()[shift:]  # noqa: E731
        assert torch.equal(ops.dropout(off(x), 0.4, 9, 11, residual=off(r), out=off(x)), want)
    a, b = x.cuda(), r.cuda()
    ops.dropout(a, 0.4, 9, 11, residual=b, out=a)
    assert torch.equal(a, want)
    a = x.cuda()
    ops.dropout(a, 0.4, 9, 11, residual=b, out=b)
    assert torch.equal(b, want)


def test_a_call_in_two_is_the_same(ops):
    """Counters are counted in fours of elements."""
    x = torch.randn(10_000, generator=torch.Generator().manual_seed(2)).cuda()
    whole = ops.dropout(x, 0.3, 42, 100)
    for cut in (4, 4000, 9996):
        parts = ops.dropout(x[:cut].contiguous(), 0.3, 42, 100), \
            ops.dropout(x[cut:].contiguous(), 0.3, 42, 100 + cut // 4)
        assert torch.equal(torch.cat(parts), whole)


def test_gradient_is_the_same_call(ops):
    """dy passes where x did, times the same factor: <dy, y(x)> is linear in x."""
    gen = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(7, 1001, generator=gen).cuda() for _ in range(2))
    y = ops.dropout(x, 0.35, 77, 3)
    dx = ops.dropout(dy, 0.35, 77, 3)
    keep = ref.dropout(x.cpu(), 0.35, 77, 3, None)[1]
    assert torch.equal(dx.cpu() != 0, keep & (dy.cpu() != 0))
    a, b = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    assert abs(a - b) <= 4 * ref.U32 * (dy.double() * y.double()).abs().sum()


def test_dropped_values_count_for_nothing(ops):
    x = torch.full((4096,), float("nan"))
    x[::2] = float("inf")
    y = ops.dropout(x.cuda(), 0.5, 5, 0, residual=torch.ones(4096).cuda()).cpu()
    keep = ref.dropout(torch.ones(4096), 0.5, 5, 0, None)[1]
    assert y[~keep].eq(1).all() and not y[keep].isfinite().any()


def test_share_and_independence(ops):
    """The share of kept elements, and of neighbours that are both kept, of a million: within five
    standard deviations."""
    n, p = 1 << 20, 0.3
    x = torch.ones(n, device="cuda")
    k = [(ops.dropout(x, p, seed, off) != 0).double()
         for seed, off in ((1, 0), (2, 0), (1, n // 4))]
    for v in k:
        assert abs(float(v.mean()) - (1 - p)) <= 5 * (p * (1 - p) / n) ** 0.5
        q = (1 - p) ** 2
        both = float((v[1:] * v[:-1]).mean())
        assert abs(both - q) <= 5 * (3 * q * (1 - q) / n) ** 0.5
    for a, b in ((0, 1), (0, 2), (1, 2)):
        q = (1 - p) ** 2
        assert abs(float((k[a] * k[b]).mean()) - q) <= 5 * (q * (1 - q) / n) ** 0.5


def test_a_graph_draws_new_numbers_by_its_counter(ops):
    x = torch.randn(3001, generator=torch.Generator().manual_seed(4))
    xc, counter = x.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda")
    ops.dropout(xc, 0.2, 6, 10, counter)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.dropout(xc, 0.2, 6, 10, counter)
        counter += 751
    seen = []
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        _check(y, x, 0.2, 6, 10 + 751 * k, None)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_nothing_to_do_and_refusals(ops):
    from splat_rendering_gb300 import pulsar as pl
    assert ops.dropout(torch.empty(0, 5, device="cuda"), 0.5, 1).shape == (0, 5)
    x = torch.zeros(8, device="cuda")
    for p in (-0.1, 1.0, 1.5, float("nan"), 1.0 - 2.0 ** -34):
        with pytest.raises(pl.PulsarError):
            ops.dropout(x, p, 1)
    with pytest.raises(TypeError):
        ops.dropout(x.half(), 0.5, 1)
    with pytest.raises(ValueError, match="contiguous"):
        ops.dropout(x[::2], 0.5, 1)
    with pytest.raises(ValueError, match="not on"):
        ops.dropout(x, 0.5, 1, counter=torch.zeros(1, dtype=torch.int64))
