"""Linear layers and dropout on tensors of more than 2^31 elements: the last rows against the same
rows alone, whose results do not depend on their place."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _fill(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g, dtype=BF16)


@pytest.mark.parametrize("rows,inputs,outputs", [(34_000_001, 64, 65), (600_001, 4096, 256)],
                         ids=["narrow", "wide"])
def test_forward_and_dx(rows, inputs, outputs):
    """(odd columns: rows at every alignment)"""
    from splat_rendering_gb300 import pulsar as pl
    ops = pl.Learner(workspace_bytes=pl.linear_workspace(rows, inputs, outputs, BF16))
    x, w = _fill((rows, inputs), 1), _fill((outputs, inputs), 2)
    w *= inputs ** -0.5
    y, _ = ops.linear(x, w, act="silu")
    for part in (slice(0, 300), slice(rows // 2, rows // 2 + 300), slice(rows - 300, rows)):
        (want, _), (bound, _) = ref.linear(x[part].cpu(), w.cpu(), None, None, "silu")
        assert not ref.outside(y[part], want, bound).any()
    dx, _, _ = ops.linear_backward(y, x, w, want=("x",))
    for part in (slice(0, 300), slice(rows - 300, rows)):
        (want, _, _), (bound, _, _) = ref.linear_backward(y[part].cpu(), x[part].cpu(), w.cpu(), None,
                                                          "none")
        assert not ref.outside(dx[part], want, bound).any()
    ops.status()
    ops.close()


@pytest.mark.parametrize("inputs,outputs", [(64, 64), (200, 48)], ids=["narrow", "wide"])
def test_sums_over_many_rows(inputs, outputs):
    """dW and db of rows that are all alike: their number times one row's."""
    from splat_rendering_gb300 import pulsar as pl
    rows = (1 << 31) // inputs + 1000
    ops = pl.Learner(workspace_bytes=pl.linear_workspace(rows, inputs, outputs, BF16))
    one, dy1 = _fill((1, inputs), 3), _fill((1, outputs), 4)
    x, dy = one.expand(rows, inputs).contiguous(), dy1.expand(rows, outputs).contiguous()
    w = _fill((outputs, inputs), 5)
    _, dw, db = ops.linear_backward(dy, x, w, want=("weight", "bias"))
    want = rows * dy1.double().T @ one.double()
    # terms of one sign: each truncated sum of up to rows / 152 of them loses at most 2 U32 of it an
    # instruction of 16, and the result is rounded
    e = (rows / 152 / 16 * 2 + 200) * ref.U32 + ref.UB
    assert ((dw.double() - want).abs() <= e * want.abs()).all()
    wb = rows * dy1.double()[0]
    assert ((db.double() - wb).abs() <= (rows / 152 / 32 + 400) * ref.U32 * wb.abs()).all()
    ops.status()
    ops.close()


def test_dropout():
    from splat_rendering_gb300 import pulsar as pl
    ops = pl.Learner(workspace_bytes=0)
    n = (1 << 31) + 4097
    x = torch.ones(n, device="cuda", dtype=BF16)
    y = ops.dropout(x, 0.25, 12345, 7)
    for at in (0, (1 << 31) - 2048, n - n % 4 - 4096):
        m = min(4096, n - at)
        want, _, bound = ref.dropout(torch.ones(m, dtype=BF16), 0.25, 12345, 7 + at // 4, None)
        assert not ref.outside(y[at:at + m], want, bound).any()
    ops.status()
    ops.close()
