"""The norm's gradients of weight and bias where there are few channels: a
block's threads then hold many parts of the same sum."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [(1, 62_579, 1, 1), (6, 446, 4, 2), (1, 5000, 4, 1), (2, 20_000, 3, 1),
                                  (1, 300_000, 2, 2)], ids=lambda c: "-".join(map(str, c)))
def test_few_channels_are_summed_as_well_as_plainly(case):
    """Root mean square over 64 inputs: no more than twice as far off as plain
    32-bit operations and sums."""
    from splat_rendering_gb300 import pulsar as pl
    N, P, C, G = case
    ops = pl.Learner(workspace_bytes=pl.group_norm_workspace(N, P, C, G))
    gen = torch.Generator(device="cuda").manual_seed(P)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    ours, plain = torch.zeros(2, dtype=torch.float64), torch.zeros(2, dtype=torch.float64)
    for _ in range(64):
        x, dy, w, b = r(N, P, C), r(N, P, C), 1 + 0.3 * r(C), 0.3 * r(C)
        _, stats = ops.group_norm(x, G, w, b, act="relu")
        _, dw, db = ops.group_norm_backward(dy, x, stats, G, w, b, "relu", want=("weight", "bias"))

        def sums(T):
            mean, rstd = (stats[..., i].to(T).reshape(N, 1, G, 1) for i in (0, 1))
            h = ((x.to(T).view(N, P, G, C // G) - mean) * rstd).view(N, P, C)
            dz = torch.where(h * w.to(T) + b.to(T) > 0, dy.to(T), 0.0)
            return (dz * h).sum((0, 1)), dz.sum((0, 1))

        exact, near = sums(torch.float64), sums(torch.float32)
        for k, (g, n, e) in enumerate(zip((dw, db), near, exact)):
            if (n.double() - e).abs().max() > 1e-3:   # a sign that differs between 32 and 64 bits
                continue
            ours[k] += float((g.double() - e).square().sum())
            plain[k] += float((n.double() - e).square().sum())
    ops.close()
    assert (ours.sqrt() <= 2 * plain.sqrt()).all(), (ours.sqrt() / plain.sqrt()).tolist()
