"""Group norm whose output is its input: the same bits as into another tensor,
for images on chip, in two launches, and in several rounds of them."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

CASES = [(2, 200, 20, 4, torch.float32), (1, 30_000, 16, 4, torch.float32),
         (1, 30_000, 3, 1, torch.bfloat16), (3, 400_000, 16, 4, torch.float32), (5, 300_001, 64, 8, torch.bfloat16)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:4])))
def test_in_place(case):
    from splat_rendering_gb300 import pulsar as pl
    N, P, C, G, T = case
    gen = torch.Generator(device="cuda").manual_seed(P)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, dy, w, b = r(N, P, C).to(T), r(N, P, C).to(T), 1 + 0.3 * r(C), 0.3 * r(C)
    ops = pl.Learner(workspace_bytes=pl.group_norm_workspace(N, P, C, G))
    y, stats = ops.group_norm(x, G, w, b, act="silu")
    want = ops.group_norm_backward(dy, x, stats, G, w, b, "silu")
    z = x.clone()
    _, again = ops.group_norm(z, G, w, b, act="silu", out=z)
    assert torch.equal(z, y) and torch.equal(again, stats)
    for k in range(2):   # dx over dy, dx over x
        ts = [dy.clone(), x.clone()]
        got = ops.group_norm_backward(*ts, stats, G, w, b, "silu", grad_x=ts[k])
        assert got[0] is ts[k] and all(map(torch.equal, got, want))
    assert ops.status() == 0
    ops.close()
