"""The orthogonalisation asks for the workspace that it uses."""
from __future__ import annotations

import pytest
import torch

SHAPES = [(8, 64, 64), (1, 3000, 10), (400, 60, 900), (2, 128, 512)]   # on chip: the matrix stays there
_ids = dict(ids=lambda c: "-".join(map(str, c)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, **_ids)
def test_on_chip_only_the_norms_parts(shape, dtype):
    """A block of the norm sums 4096 elements at least and leaves 16 bytes."""
    from splat_rendering_gb300 import build, pulsar as pl
    build.build()
    B, m, n = shape
    need = pl.orthogonalize_workspace(B, m, n, dtype)
    assert 0 < need <= B * 16 * (m * n // 4096 + 1) + 256


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES + [(3, 200, 300)], **_ids)
@pytest.mark.parametrize("steps", [0, 5])
def test_the_workspace_is_enough(shape, dtype, steps):
    """The same bits as with room to spare, and nothing less is taken."""
    from splat_rendering_gb300 import pulsar as pl
    B, m, n = shape
    need = pl.orthogonalize_workspace(B, m, n, dtype)
    g = torch.randn(*shape, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    exact, roomy, short = (pl.Learner(workspace_bytes=v) for v in (need, need + (1 << 26), need - 1))
    assert torch.equal(exact.orthogonalize(g, steps=steps), roomy.orthogonalize(g, steps=steps))
    with pytest.raises(pl.PulsarError, match="workspace"):
        short.orthogonalize(g, steps=steps)
    for o in (exact, roomy, short):
        o.status()
        o.close()
