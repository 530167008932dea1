"""Group norm of a large image whose first rows are far from the rest (a
border): the statistics joined from the blocks' parts, the first of which is
no guide to the others."""
from __future__ import annotations

import pytest
import torch

import learn_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("border", [4096, 20_000, 1 << 17])
def test_two_constants(border, dtype):
    """Pixels of 8, then of 0: every part's own statistics are exact or nearly
    so, and what is left are the joins.  About the common mean, a sum over the
    blocks (fewer than 512: 16 a lane, 5 levels of the warp, the shares' two
    roundings) is off by 24 U32 of its terms' magnitudes, all positive for the
    variance; a straddling block's own second moment by less.  The square
    root halves that and adds 4 U32.  The mean is off by 24 U32 of the mean
    distance from it, and rounded."""
    from splat_rendering_gb300 import pulsar as pl
    P, C, G = 1 << 20, 16, 4
    x = torch.zeros(1, P, C, dtype=dtype, device="cuda")
    x[:, :border] = 8.0
    ops = pl.Learner(workspace_bytes=pl.group_norm_workspace(1, P, C, G))
    _, stats = ops.group_norm(x, G, eps=0.0)
    f = border / P
    mean, rstd = 8.0 * f, (64.0 * f * (1 - f)) ** -0.5
    got = stats[0].double().cpu()
    assert (got[:, 1] / rstd - 1).abs().max() <= 16 * ref.U32
    assert (got[:, 0] - mean).abs().max() <= 24 * ref.U32 * 16.0 * f * (1 - f) + ref.U32 * mean
    ops.close()
