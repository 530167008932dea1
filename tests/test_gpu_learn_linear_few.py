"""Layers of a few outputs, at the sizes where their kernels divide rows and inputs differently."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref
from test_gpu_learn_linear import TYPES, _cuda, _inputs, _inside, _near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=1 << 29)
    yield o
    assert o.status() == 0
    o.close()


# rows (few, a block's, more than one chunk of a block), inputs (loads of 16, 8, 4 and 2 bytes; one
# lane to a row, several, all, several loads to a lane; a block of columns, several; the most and one
# more), outputs (the most and one more)
CASES = [(9, 1, 1), (33, 2, 3), (300, 3, 4), (301, 7, 2), (1025, 8, 1), (77, 31, 4), (77, 33, 4),
         (500, 52, 3), (129, 64, 4), (130, 96, 1), (200, 130, 2), (64, 255, 4), (64, 256, 4),
         (64, 257, 3), (40, 1000, 1), (41, 2048, 1), (41, 2048, 4), (41, 2049, 1), (600, 2046, 4),
         (400, 40, 5), (700_001, 3, 3), (70_001, 50, 1), (5000, 1026, 2), (40_000, 128, 4)]


@pytest.mark.parametrize("name", ["none", "silu", "relu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_few_outputs(ops, case, dtype, name):
    M, K, N = case
    x, w, b, r, dy = _inputs(M, K, N, TYPES[dtype], 700 + M + K + N)
    xc, wc, bc, rc, dyc = _cuda(x, w, b, r, dy)
    y, z = ops.linear(xc, wc, bc, rc, name, want_pre=True)
    (y_want, z_want), (e_y, e_z) = ref.linear(x, w, b, r, name)
    _inside(z, z_want, e_z, "z")
    _inside(y, y_want, e_y, "y")
    _near(z, z_want, "z")
    assert torch.equal(ops.linear(xc, wc, bc, rc, name)[0], y)
    over = rc.clone()
    assert torch.equal(ops.linear(xc, wc, bc, over, name, out=over)[0], y)
    got = ops.linear_backward(dyc, xc, wc, z, name)
    want, bounds = ref.linear_backward(dy, x, w, z.cpu(), name)
    for g, v, e, what in zip(got, want, bounds, ("dx", "dw", "db")):
        _inside(g, v, e, what)
        _near(g, v, what)
    for i, one in enumerate(("x", "weight", "bias")):   # each alone, to the same bits
        alone = ops.linear_backward(dyc, xc, wc, z, name, want=(one,))
        assert [a is not None for a in alone] == [j == i for j in range(3)]
        assert torch.equal(alone[i], got[i]), one


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("case", [(50, 64, 3), (300, 200, 4)], ids=lambda c: "-".join(map(str, c)))
def test_tensors_that_begin_anywhere(ops, case, off, dtype):
    """Narrower loads where tensors do not begin on 16 bytes, to the same results; nothing beyond
    the outputs is written, and what lies behind the inputs is not read into them."""
    M, K, N = case
    t = TYPES[dtype]
    x, w, b, r, dy = _cuda(*_inputs(M, K, N, t, 800))

    def moved(v):
        room = torch.full((v.numel() + 32,), float("nan"), dtype=v.dtype, device="cuda")
        room[off:off + v.numel()] = v.reshape(-1)
        return room, room[off:off + v.numel()].view(v.shape)

    (rx, xm), (rw, wm), (ry, dym) = moved(x), moved(w), moved(dy)
    room, out = moved(r)
    y, z = ops.linear(xm, wm, b, None, "silu", want_pre=True, out=out)
    (y_want, _), (e_y, _) = ref.linear(x.cpu(), w.cpu(), b.cpu(), None, "silu")
    _inside(y, y_want, e_y, "y")
    assert room[:off].isnan().all() and room[off + out.numel():].isnan().all()
    room, gx = moved(x)
    got = ops.linear_backward(dym, xm, wm, z, "silu", grad_x=gx)
    want, bounds = ref.linear_backward(dy.cpu(), x.cpu(), w.cpu(), z.cpu(), "silu")
    for g, v, e, what in zip(got, want, bounds, ("dx", "dw", "db")):
        _inside(g, v, e, what)
    assert room[:off].isnan().all() and room[off + gx.numel():].isnan().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(3000, 40, 3), (900, 512, 512), (2000, 100, 5)],
                         ids=lambda c: "-".join(map(str, c)))
def test_captured_and_replayed(ops, case, dtype):
    """A captured step reads its tensors when it is replayed, and leaves what a call leaves."""
    x, w, b, _, dy = _cuda(*_inputs(*case, TYPES[dtype], 900))
    step = lambda: (ops.linear(x, w, b, act="relu", want_pre=True),  # noqa: E731
                    ops.linear_backward(dy, x, w))
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        (y, z), grads = step()
    x.mul_(-0.5)
    dy.mul_(2)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    (y2, z2), grads2 = step()
    assert torch.equal(y, y2) and torch.equal(z, z2)
    assert all(torch.equal(p, q) for p, q in zip(grads, grads2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        (y3, _), grads3 = step()
    side.synchronize()
    assert torch.equal(y, y3) and all(torch.equal(p, q) for p, q in zip(grads, grads3))
