"""The linear layer's forms at the sizes where one takes over from another, its extreme sizes, and
calls that share tensors."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref
from test_gpu_learn_linear import TYPES, _cuda, _inputs, _inside, _near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=1 << 30)
    yield o
    assert o.status() == 0
    o.close()


# few rows and one more; narrow layers of one block of outputs, of eight, and one more; a
# contraction of 64 and 128 and one more; 64 and 128 outputs, backward, and one more; one row of
# tiles and two; one output of many inputs; parts of a contraction and none
CASES = [
    (6, 1001, 70), (7, 64, 33), (8, 4096, 130), (9, 4096, 130), (9, 40, 24),
    (300, 64, 512), (300, 64, 513), (300, 100, 1024), (300, 100, 1025), (300, 128, 200),
    (300, 129, 200), (400, 64, 65), (400, 65, 64), (400, 128, 129), (400, 129, 128),
    (128, 300, 300), (129, 300, 300), (256, 512, 256), (257, 520, 264), (130, 4096, 1),
    (50, 1, 1100), (300, 3, 1500), (3000, 2, 1), (20, 20_000, 40), (20_000, 200, 40),
    (12, 65_536, 3), (12, 3, 65_536), (2, 65_536, 2),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forms(ops, case, dtype):
    M, K, N = case
    x, w, b, r, dy = _inputs(M, K, N, TYPES[dtype], 300 + M + K + N)
    xc, wc, bc, rc, dyc = _cuda(x, w, b, r, dy)
    y, z = ops.linear(xc, wc, bc, rc, "silu", want_pre=True)
    (y_want, z_want), (e_y, e_z) = ref.linear(x, w, b, r, "silu")
    _inside(z, z_want, e_z, "z")
    _inside(y, y_want, e_y, "y")
    _near(z, z_want, "z")
    got = ops.linear_backward(dyc, xc, wc, z, "silu")
    want, bounds = ref.linear_backward(dy, x, w, z.cpu(), "silu")
    for g, v, e, what in zip(got, want, bounds, ("dx", "dw", "db")):
        _inside(g, v, e, what)
        _near(g, v, what)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(5, 70, 50), (900, 40, 64), (900, 41, 63), (40, 4096, 64),
                                  (600, 200, 300)], ids=lambda c: "-".join(map(str, c)))
def test_the_result_over_its_residual(ops, case, dtype):
    """In every form, with the residual's bits read before they are written."""
    x, w, b, r, _ = _cuda(*_inputs(*case, TYPES[dtype], 401))
    want, _ = ops.linear(x, w, b, r, "relu")
    ops.linear(x, w, b, r, "relu", out=r)
    assert torch.equal(r, want)


def test_one_tensor_as_several_inputs(ops):
    """x is the weight, the residual and the incoming gradient: all are only read."""
    for n in (64, 200):
        x = torch.randn(n, n, generator=torch.Generator().manual_seed(n)).cuda()
        keep = x.clone()
        y, _ = ops.linear(x, x, None, x)
        assert torch.equal(x, keep)
        (want, _), (bound, _) = ref.linear(x.cpu(), x.cpu(), None, x.cpu(), "none")
        _inside(y, want, bound, "y")
        got = ops.linear_backward(x, x, x)
        want, bounds = ref.linear_backward(x.cpu(), x.cpu(), x.cpu(), None, "none")
        for g, v, e, what in zip(got, want, bounds, ("dx", "dw", "db")):
            _inside(g, v, e, what)
        assert torch.equal(x, keep)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(5, 70, 50), (900, 40, 64), (901, 41, 63), (601, 200, 303)],
                         ids=lambda c: "-".join(map(str, c)))
def test_nothing_else_is_written(ops, case, dtype):
    """Outputs inside larger buffers: what lies before and behind them stays."""
    M, K, N = case
    T = TYPES[dtype]
    x, w, b, r, dy = _cuda(*_inputs(M, K, N, T, 501))

    def inside(shape, dt):
        n = shape.numel()
        buf = torch.full((n + 256,), 7.0, dtype=dt, device="cuda")
        return buf, buf[128:128 + n].view(shape)

    bufs = [inside(s, t) for s, t in ((r.shape, T), (r.shape, T), (x.shape, T), (w.shape, T),
                                      (b.shape, torch.float32))]
    (_, y), (_, z), (_, gx), (_, gw), (_, gb) = bufs
    ops.linear(x, w, b, r, "silu", out=y, pre=z)
    ops.linear_backward(dy, x, w, z, "silu", grad_x=gx, grad_weight=gw, grad_bias=gb)
    for buf, t in bufs:
        assert buf[:128].eq(7).all() and buf[128 + t.numel():].eq(7).all()
    assert torch.equal(y, ops.linear(x, w, b, r, "silu")[0])


def test_rows_do_not_depend_on_their_place(ops):
    """Rows of one call, and the same rows of another of the same form, have the same bits."""
    for T in TYPES.values():
        x, w, b, _, _ = _cuda(*_inputs(5000, 64, 64, T, 601))
        y, _ = ops.linear(x, w, b, act="silu")
        part, _ = ops.linear(x[1000:2111].contiguous(), w, b, act="silu")
        assert torch.equal(part, y[1000:2111])
