"""Group norm of batches larger than the L2, taken several images at a time:
the rounds reuse their workspace, and the last one is shorter."""
from __future__ import annotations

import pytest
import torch

import learn_reference as ref

pytestmark = pytest.mark.gpu


def _inside(got, want, bound):
    return not ref.outside(got, want.cpu(), bound.cpu()).any()


# rounds of two images and one, forward; then of two and one backward; five of 16 bits by twos
@pytest.mark.parametrize("case", [(3, 1 << 20, 16, 4, torch.float32), (3, 400_000, 16, 4, torch.float32),
                                  (5, 300_001, 64, 8, torch.bfloat16)],
                         ids=lambda c: "-".join(map(str, c[:4])))
def test_rounds(case):
    from splat_rendering_gb300 import pulsar as pl
    N, P, C, G, T = case
    gen = torch.Generator(device="cuda").manual_seed(P)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    # every image has its own scale and mean
    x = torch.cat([r(1, P, C) * (1 + i) + r(C) + i for i in range(N)]).to(T)
    dy = torch.cat([r(1, P, C) / (1 + i) for i in range(N)]).to(T)
    w, b = 1 + 0.3 * r(C), 0.3 * r(C)
    ops = pl.Learner(workspace_bytes=pl.group_norm_workspace(N, P, C, G))
    y, stats = ops.group_norm(x, G, w, b, act="silu")
    got = ops.group_norm_backward(dy, x, stats, G, w, b, "silu")
    sums = []
    for i in range(N):
        one = slice(i, i + 1)
        want, s_want, e_y, e_s = ref.group_norm(x[one], G, w, b, 1e-5, "silu")
        assert _inside(stats[one], s_want, e_s), i
        assert _inside(y[one], want, e_y), i
        del want, e_y
        want, bounds = ref.group_norm_backward(dy[one], x[one], stats[one], G, w, b, "silu")
        assert _inside(got[0][one], want[0], bounds[0]), i
        sums.append((want[1], want[2], bounds[1], bounds[2]))
    dw, db, e_w, e_b = (sum(t) for t in zip(*sums))
    assert _inside(got[1], dw, e_w) and _inside(got[2], db, e_b)
    assert ops.status() == 0
    ops.close()
