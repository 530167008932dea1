"""Outputs of a linear layer or of dropout that share memory with what they may not are refused, and
nothing is written; those that may be an input are that input or apart from it."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
K = 64   # (square tensors, so that each could be any other)


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=1 << 24)
    yield o
    assert o.status() == 0
    o.close()


def _tensors(count, rows=K):
    g = torch.Generator().manual_seed(51)
    return [torch.randn(rows, K, generator=g).cuda() for _ in range(count)]


def test_linear_refuses(ops):
    from splat_rendering_gb300 import pulsar as pl
    x, w, r, y, z = _tensors(5)
    keep = [t.clone() for t in (x, w, r, y, z)]
    b = torch.zeros(K, device="cuda")
    for kw in (dict(out=x), dict(out=w), dict(pre=x), dict(pre=w), dict(pre=r), dict(out=y, pre=y),
               dict(out=r, pre=r)):
        with pytest.raises(pl.PulsarError, match="argument"):
            ops.linear(x, w, b, r, "silu", **kw)
    room = torch.zeros(3 * K * K, device="cuda")
    at = lambda n: room[n:n + K * K].view(K, K)  # noqa: E731
    for kw in (dict(residual=at(0), out=at(4)), dict(residual=at(8), out=at(0)), dict(out=at(0), pre=at(K * K - 1))):
        with pytest.raises(pl.PulsarError, match="argument"):
            ops.linear(x, w, b, **kw)
    with pytest.raises(pl.PulsarError, match="argument"):
        ops.linear(x, w, room[5:5 + K], out=at(0))
    for t, k in zip((x, w, r, y, z), keep):
        assert torch.equal(t, k)
    assert room.eq(0).all()
    # side by side is apart, and the residual's own place is allowed
    want, _ = ops.linear(x, w, b, r)
    ops.linear(x, w, b, r, out=at(0), pre=at(K * K))
    assert torch.equal(at(0), want)
    ops.linear(x, w, b, r, out=r)
    assert torch.equal(r, want)


def test_linear_backward_refuses(ops):
    from splat_rendering_gb300 import pulsar as pl
    dy, x, w, z, g = _tensors(5)
    keep = [t.clone() for t in (dy, x, w, z)]
    row = lambda t: t.view(-1)[K:2 * K]  # noqa: E731
    for kw in (dict(grad_x=dy), dict(grad_x=x), dict(grad_x=w), dict(grad_x=z), dict(grad_weight=w),
               dict(grad_weight=x), dict(grad_weight=dy), dict(grad_weight=z), dict(grad_x=g, grad_weight=g),
               dict(grad_bias=row(dy)), dict(grad_bias=row(z)), dict(grad_x=g, grad_bias=row(g)),
               dict(grad_weight=g, grad_bias=row(g))):
        with pytest.raises(pl.PulsarError, match="argument"):
            ops.linear_backward(dy, x, w, z, "silu", want=(), **kw)
    for t, k in zip((dy, x, w, z), keep):
        assert torch.equal(t, k)
    # inputs may be one another, and an empty tensor lies nowhere
    ops.linear_backward(x, x, x, x, "silu")
    none = x[:0]
    _, gw, _ = ops.linear_backward(none, none, w, grad_weight=x)
    assert gw.eq(0).all()


def test_dropout_refuses(ops):
    from splat_rendering_gb300 import pulsar as pl
    room = torch.randn(4000, generator=torch.Generator().manual_seed(52)).cuda()
    keep, n = room.clone(), 1000
    x, r = room[:n], room[2000:2000 + n]
    counter = torch.zeros(8, dtype=torch.int64, device="cuda")
    for out in (room[1:1 + n], room[n - 1:2 * n - 1], room[1996:1996 + n], room[2001:2001 + n]):
        with pytest.raises(pl.PulsarError, match="argument"):
            ops.dropout(x, 0.5, 1, residual=r, out=out)
    with pytest.raises(pl.PulsarError, match="argument"):
        ops.dropout(x[:2], 0.5, 1, counter=counter[:1], out=counter.view(torch.float32)[:2])
    assert torch.equal(room, keep)
    want = ops.dropout(x, 0.5, 1, residual=r)
    assert torch.equal(ops.dropout(x, 0.5, 1, residual=r, out=room[n:2 * n]), want)
    assert torch.equal(ops.dropout(x, 0.5, 1, residual=r, out=r), want)
