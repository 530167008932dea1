"""Infinities and NaNs through every form of the linear layer and of its gradients: they stay in
their rows and columns, and no activation hides them."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref
from test_gpu_learn_linear import TYPES, _cuda, _inputs, _inside

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")

# few rows, a narrow layer of whole and of other rows, wide layers of small tiles, of pairs, and of
# both with rows that are no whole vectors, few outputs of few and of many inputs
CASES = [(5, 70, 50), (8, 64, 4), (300, 64, 64), (301, 41, 63), (100, 200, 72), (300, 200, 303),
         (700, 512, 2100), (300, 40, 3), (300, 300, 3), (300, 300, 1)]


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=1 << 29)
    yield o
    assert o.status() == 0
    o.close()


@pytest.mark.parametrize("name", ["none", "silu", "relu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward(ops, case, dtype, name):
    """Where z's sum is a NaN y is one; where it is +inf, y is that or a NaN; where it is -inf, y is
    a NaN or what the activation makes of it; everywhere else y is the finite value."""
    M, K, N = case
    x, w, b, r, _ = _inputs(M, K, N, TYPES[dtype], 11)
    (want, z), (bound, _) = ref.linear(x, w, b, r, name)
    x[0, K // 2], x[1, 0], x[2, K - 1] = INF, NAN, -INF
    if N > 1:
        w[N - 1, K // 3] = -INF
    z = x.double() @ w.double().T + b.double()
    y, pre = (t.cpu() for t in ops.linear(*_cuda(x, w, b, r), name, want_pre=True))
    assert not pre[~z.isfinite()].isfinite().any()
    for t in (y, pre):
        assert t[z.isnan()].isnan().all()
        up = t[z == INF]
        assert (up.isnan() | (up == INF)).all()
    down = y[z == -INF]
    least = r[z == -INF] if name == "relu" else torch.full_like(down, -INF)
    assert (down.isnan() | (down == least)).all()
    fine = z.isfinite()
    assert fine.any() and not ref.outside(y[fine], want[fine], bound[fine]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_gradients_of_relu(ops, case, dtype):
    """dy passes where z is +inf or a NaN (a sum with an infinity), and not where it is -inf."""
    M, K, N = case
    x, w, _, z, dy = _inputs(M, K, N, TYPES[dtype], 12)
    z[0, 0], z[1, 0], z[2, 0], z[1, N - 1] = INF, NAN, -INF, NAN
    got = ops.linear_backward(*_cuda(dy, x, w, z), "relu")
    open_ = z.clone()
    open_[z.isnan()] = 1.0
    want, bounds = ref.linear_backward(dy, x, w, open_, "relu")
    for g, v, e, what in zip(got, want, bounds, ("dx", "dw", "db")):
        _inside(g, v, e, what)


@pytest.mark.parametrize("name", ["none", "relu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_gradients_of_nonfinite_rows(ops, case, dtype, name):
    """An infinity or a NaN in dy reaches its row of dx, its row of dW and its sum in db; in x, its
    column of dW; nothing else.  Behind a closed ReLU it reaches nothing."""
    M, K, N = case
    x, w, _, z, dy = _inputs(M, K, N, TYPES[dtype], 13)
    z = z.abs() + 0.5
    z[2, 0] = -1.0
    clean = dy.clone()
    clean[0, 0] = clean[1, N - 1] = 0.0
    want, bounds = ref.linear_backward(clean, x, w, z, name)
    dy[0, 0], dy[1, N - 1], dy[2, 0] = INF, NAN, (NAN if name == "relu" else dy[2, 0])
    if name == "relu":
        clean[2, 0] = 0.0
        want, bounds = ref.linear_backward(clean, x, w, z, name)
    dx, dw, db = (t.cpu() for t in ops.linear_backward(*_cuda(dy, x, w, z), name))
    assert not dx[:2].isfinite().any() and not dw[[0, N - 1]].isfinite().any()
    assert not db[[0, N - 1]].isfinite().any()
    for g, v, e in ((dx[2:], want[0][2:], bounds[0][2:]), (dw[1:N - 1], want[1][1:N - 1], bounds[1][1:N - 1]),
                    (db[1:N - 1], want[2][1:N - 1], bounds[2][1:N - 1])):
        assert not ref.outside(g, v, e).any()
    x[1, K // 2] = NAN
    want, bounds = ref.linear_backward(clean, x, w, z, name)
    dx, dw, db = (t.cpu() for t in ops.linear_backward(*_cuda(clean, x, w, z), name))
    other = torch.arange(K) != K // 2
    # (row 1 of dy has a zero in its last column: there 0 * NaN is NaN too)
    assert dw[:, K // 2].isnan().all()
    assert not ref.outside(dw[:, other], want[1][:, other], bounds[1][:, other]).any()
    assert not ref.outside(dx, want[0], bounds[0]).any()
    assert not ref.outside(db, want[2], bounds[2]).any()
