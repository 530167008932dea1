"""The linear layer on operands near the smallest numbers: in 32 bits an operand's three parts of
16 bits end at 2^-133, so that it is off by at most half of that (and by nothing above 2^-110)."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref
from test_gpu_learn_linear import TYPES, _cuda, _inside, _near

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -134


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=1 << 28)
    yield o
    assert o.status() == 0
    o.close()


@pytest.mark.parametrize("scale", [2.0 ** -105, 2.0 ** -118, 2.0 ** -129])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(5, 70, 50), (200, 40, 64), (201, 41, 63), (300, 200, 303)],
                         ids=lambda c: "-".join(map(str, c)))
def test_small_operands(ops, case, dtype, scale):
    """x and dy below the least normal number times weights as much above one: nothing that is
    representable is taken for zero."""
    M, K, N = case
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(511)
    draw = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, dy = (draw(M, K) * scale).to(t), (draw(M, N) * scale).to(t)
    big = min(1 / scale, 2.0 ** 120)
    w = (draw(N, K) * big).to(t)
    xc, wc, dyc = _cuda(x, w, dy)
    y, _ = ops.linear(xc, wc)
    (want, _), (bound, _) = ref.linear(x, w, None, None, "none")
    lost = LEAST if dtype == "f32" else 0.0
    _inside(y, want, bound + lost * w.double().abs().sum(1), "y")
    gx, _, _ = ops.linear_backward(dyc, xc, wc, want=("x",))
    (want, _, _), (bound, _, _) = ref.linear_backward(dy, x, w, None, "none")
    _inside(gx, want, bound + lost * w.double().abs().sum(0), "dx")
    if scale > 2.0 ** -110:
        _near(y, (x.double() @ w.double().T), "y")
    # the weights' gradient of small rows and large gradients
    up = (draw(M, N) * big).to(t)
    _, gw, gb = ops.linear_backward(up.cuda(), xc, wc, want=("weight", "bias"))
    (_, want, want_b), (_, bound, bound_b) = ref.linear_backward(up, x, w, None, "none")
    _inside(gw, want, bound + lost * up.double().abs().sum(0)[:, None], "dw")
    _inside(gb, want_b, bound_b, "db")
