"""Gradients of a weight over many rows in 16 bits: sums that the tensor cores truncate are drained
every 2^14 rows, so that what they lose does not grow with the rows."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
DRAIN = 1 << 14   # rows


def _one(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((1, n), device="cuda", generator=g, dtype=BF16)


def _alike(rows, inputs, outputs, want=("weight", "bias")):
    """dW of rows that are all alike, so that all of a sum's terms have one sign, by the number of
    rows: each of a piece's DRAIN / 16 instructions truncates at most 2 U32 of its sum, the pieces and
    the parts are added in float32, and the result is rounded."""
    from splat_rendering_gb300 import pulsar as pl
    ops = pl.Learner(workspace_bytes=pl.linear_workspace(rows, inputs, outputs, BF16))
    one, dy1 = _one(inputs, 3), _one(outputs, 4)
    x, dy = one.expand(rows, inputs).contiguous(), dy1.expand(rows, outputs).contiguous()
    w = _one(inputs, 5).expand(outputs, inputs).contiguous()
    _, dw, _ = ops.linear_backward(dy, x, w, want=want)
    exact = rows * dy1.double().T @ one.double()
    e = (2 * DRAIN / 16 + rows / DRAIN + 304 + 4) * ref.U32 + ref.UB
    bad = (dw.double() - exact).abs() > e * exact.abs()
    assert not bad.any(), (int(bad.sum()), float(((dw.double() - exact) / exact).abs().max()), e)
    ops.status()
    ops.close()


@pytest.mark.parametrize("rows,inputs,outputs", [(1 << 21, 2560, 1024), ((1 << 21) + 77, 256, 9728),
                                                 (4_000_001, 520, 264)],
                         ids=["one-part", "one-part-oblong", "parts"])
def test_wide(rows, inputs, outputs):
    _alike(rows, inputs, outputs)


@pytest.mark.parametrize("rows,inputs,outputs", [(3_000_001, 300, 301), (700_003, 129, 1200), (200_000, 2560, 1024)])
def test_wide_against_64_bits(rows, inputs, outputs):
    """Pieces of rows that differ, and a last one that is not whole."""
    from splat_rendering_gb300 import pulsar as pl
    ops = pl.Learner(workspace_bytes=pl.linear_workspace(rows, inputs, outputs, BF16))
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dy, w = (torch.randn(s, device="cuda", generator=g, dtype=BF16)
                for s in ((rows, inputs), (rows, outputs), (outputs, inputs)))
    _, dw, _ = ops.linear_backward(dy, x, w, want=("weight",))
    want = torch.zeros(outputs, inputs, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for at in range(0, rows, 200_000):
        a, b = dy[at:at + 200_000].double(), x[at:at + 200_000].double()
        want += a.T @ b
        size += a.abs().T @ b.abs()
    bound = (2 * DRAIN / 16 + rows / DRAIN + 304 + 4) * ref.U32 * size
    assert not ref.outside(dw, want.cpu(), bound.cpu()).any()
    ops.status()
    ops.close()


@pytest.mark.parametrize("want", [("weight", "bias"), ("x", "weight", "bias")], ids=["first", "inner"])
@pytest.mark.parametrize("rows,inputs,outputs", [(1 << 25, 64, 64), ((1 << 23) + 99, 128, 100)])
def test_narrow(rows, inputs, outputs, want):
    _alike(rows, inputs, outputs, want)


@pytest.mark.parametrize("rows", [152 * 128 * 128, 152 * 128 * 128 + 1, 3 * 152 * 128 * 128 - 500])
@pytest.mark.parametrize("inputs,outputs", [(40, 24), (33, 17), (100, 128), (16, 128)])
def test_narrow_against_64_bits(rows, inputs, outputs):
    """Whole pieces, one tile of another, and several."""
    from splat_rendering_gb300 import pulsar as pl
    ops = pl.Learner(workspace_bytes=pl.linear_workspace(rows, inputs, outputs, BF16))
    g = torch.Generator(device="cuda").manual_seed(8)
    x, dy, w = (torch.randn(s, device="cuda", generator=g, dtype=BF16)
                for s in ((rows, inputs), (rows, outputs), (outputs, inputs)))
    dx, dw, db = ops.linear_backward(dy, x, w)
    alone = ops.linear_backward(dy, x, w, want=("weight",))[1]
    assert torch.equal(dw, alone)
    want = torch.zeros(outputs, inputs, dtype=torch.float64, device="cuda")
    size, sums, sizes = torch.zeros_like(want), 0.0, 0.0
    for at in range(0, rows, 500_000):
        a, b = dy[at:at + 500_000].double(), x[at:at + 500_000].double()
        want += a.T @ b
        size += a.abs().T @ b.abs()
        sums, sizes = sums + a.sum(0), sizes + a.abs().sum(0)
    bound = (2 * DRAIN / 16 + rows / DRAIN + 304 + 4) * ref.U32 * size
    assert not ref.outside(dw, want.cpu(), bound.cpu()).any()
    assert not ref.outside(db, sums.cpu(), ((rows / 152 / 32 + 400) * ref.U32 * sizes).cpu()).any()
    for part in (slice(0, 200), slice(rows - 200, rows)):
        (v, _, _), (e, _, _) = ref.linear_backward(dy[part].cpu(), x[part].cpu(), w.cpu(), None, "none")
        assert not ref.outside(dx[part], v, e).any()
    ops.status()
    ops.close()


@pytest.mark.parametrize("rows,inputs,outputs", [(2 * 152 * 128 * 128 + 5, 64, 64), (200_000, 2560, 1024),
                                                 (1_000_000, 300, 301)])
def test_captured_and_on_two_streams(rows, inputs, outputs):
    """A captured call, replayed beside another handle's on another stream, leaves an eager call's bits."""
    from splat_rendering_gb300 import pulsar as pl
    g = torch.Generator(device="cuda").manual_seed(9)
    x, dy, w = (torch.randn(s, device="cuda", generator=g, dtype=BF16)
                for s in ((rows, inputs), (rows, outputs), (outputs, inputs)))
    a, b = (pl.Learner(workspace_bytes=pl.linear_workspace(rows, inputs, outputs, BF16)) for _ in range(2))
    want = a.linear_backward(dy, x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = a.linear_backward(dy, x, w)
    side = torch.cuda.Stream()
    for _ in range(2):
        graph.replay()
        with torch.cuda.stream(side):
            other = b.linear_backward(dy, x, w)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) and torch.equal(r, q) for p, q, r in zip(got, want, other))
    for o in (a, b):
        assert o.status() == 0
        o.close()
