"""Linear layers on a handle with just the workspace that they ask for, tensors at any alignment."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref
from test_gpu_learn_linear import TYPES, _cuda, _inputs, _inside

pytestmark = pytest.mark.gpu

# narrow layers, one block of outputs and several; few outputs, of which the products take some; wide
# layers, of one part and of several, and those that are narrow one way only
CASES = [(300, 64, 64), (301, 41, 63), (500, 128, 100), (300, 7, 900), (300, 96, 4), (300, 1000, 2),
         (70, 512, 4), (3000, 1024, 3), (300, 200, 303), (40, 4096, 200), (2000, 100, 513),
         (20_000, 129, 5), (9, 3000, 40), (8, 300, 70)]


def _moved(t, off):
    """The tensor `off` elements from where memory begins, with NaNs around it."""
    room = torch.full((t.numel() + 64,), float("nan"), dtype=t.dtype, device="cuda")
    room[off:off + t.numel()] = t.reshape(-1)
    return room[off:off + t.numel()].view(t.shape)


@pytest.mark.parametrize("off", [0, 1, 2, 4, 7])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_just_enough(case, dtype, off):
    from splat_rendering_gb300 import pulsar as pl
    M, K, N = case
    T = TYPES[dtype]
    x, w, b, r, dy = _inputs(M, K, N, T, 31)
    ops = pl.Learner(workspace_bytes=pl.linear_workspace(M, K, N, T))
    xm, wm, rm, dm = (_moved(t, off) for t in (x, w, r, dy))
    y, z = ops.linear(xm, wm, b.cuda(), rm, "silu", want_pre=True)
    (y_want, z_want), (e_y, e_z) = ref.linear(x, w, b, r, "silu")
    _inside(z, z_want, e_z, "z")
    _inside(y, y_want, e_y, "y")
    got = ops.linear_backward(dm, xm, wm, _moved(z, off), "silu")
    want, bounds = ref.linear_backward(dy, x, w, z.cpu(), "silu")
    for g, v, e, what in zip(got, want, bounds, ("dx", "dw", "db")):
        _inside(g, v, e, what)
    assert ops.status() == 0
    ops.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_rows_ask_for_none(dtype):
    from splat_rendering_gb300 import pulsar as pl
    T = TYPES[dtype]
    ops = pl.Learner(workspace_bytes=0)
    for M in (1, 8):
        x, w, b, _, _ = _inputs(M, 500, 200, T, 32)
        y, _ = ops.linear(*_cuda(x, w, b), act="relu")
        (want, _), (bound, _) = ref.linear(x, w, b, None, "relu")
        _inside(y, want, bound, "y")
    x, w, b, _, _ = _cuda(*_inputs(9, 500, 200, T, 32))
    with pytest.raises(pl.PulsarError, match="workspace"):
        ops.linear(x, w, b)
    ops.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(9, 1, 8), (129, 64, 64), (1000, 41, 63), (5000, 128, 300)],
                         ids=lambda c: "-".join(map(str, c)))
def test_narrow_rows_are_the_same_wherever_they_begin(case, dtype):
    """The same bits, and nothing from around x in them."""
    from splat_rendering_gb300 import pulsar as pl
    M, K, N = case
    T = TYPES[dtype]
    x, w, b, r, _ = _cuda(*_inputs(M, K, N, T, 33))
    ops = pl.Learner(workspace_bytes=pl.linear_workspace(M, K, N, T))
    y, _ = ops.linear(x, w, b, r, "relu")
    for off in range(1, 9):
        assert torch.equal(ops.linear(_moved(x, off), w, b, r, "relu")[0], y), off
    ops.close()
