"""The bias' gradient: a million rows whose sum cancels.

A chain of n float32 additions of values that are independent and centred has partial sums that grow
with the root of their number, and each addition is off by at most U32 / sqrt(3) (rms) of its own: of
rows / n such chains the sum is off by U32 sqrt(n / 6) of its norm.  A thread of a narrow layer adds
four rows, and then the fours of its tiles, two a tile, to a chain: 92 for 46 tiles; what follows
(the threads' and the CTAs' sums, added in some 30 steps) is as a chain of 30 at most."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inputs,outputs,act", [(64, 64, "none"), (64, 64, "silu"), (41, 63, "none"), (16, 64, "relu")])
def test_sums_that_cancel(inputs, outputs, act):
    from splat_rendering_gb300 import pulsar as pl
    rows = 1 << 20
    ops = pl.Learner(workspace_bytes=pl.linear_workspace(rows, inputs, outputs, torch.float32))
    g = torch.Generator(device="cuda").manual_seed(21)
    x, dy, w, z = (torch.randn(s, device="cuda", generator=g)
                   for s in ((rows, inputs), (rows, outputs), (outputs, inputs), (rows, outputs)))
    _, _, db = ops.linear_backward(dy, x, w, z, act, want=("bias",))
    dz = dy.double()
    if act != "none":
        dz = dz * ref.act_grad(z.double(), act)
    want = dz.sum(0)
    e = float((db.double() - want).norm() / want.norm())
    assert e <= ref.U32 * ((92 + 30) / 6) ** 0.5, e
    ops.status()
    ops.close()
