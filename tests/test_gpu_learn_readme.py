"""The README's training step of the learned parts, as it stands there, against autograd in 64 bits."""
from __future__ import annotations

import os
import re

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _step():
    blocks = re.findall(r"```python\n(.*?)```", open(README).read(), flags=re.S)
    (code,) = [b for b in blocks if "ops.linear_backward" in b]
    return code


def test_the_step_computes_its_gradients():
    from splat_rendering_gb300 import pulsar as pl
    g = torch.Generator().manual_seed(41)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    H, W, n, rows = 20, 30, 50, 11
    cpu = dict(image=r(H, W, 16), gamma=1 + 0.2 * r(16), beta=0.2 * r(16), weight=r(64, 16) / 4,
               bias=0.2 * r(64), weight2=r(16, 64) / 8, bias2=0.2 * r(16), gout=r(1, H, W, 16))
    space = dict(pl=pl, torch=torch, n=n, rows=rows, H=H, W=W, seed=77, offset=5,
                 codebook=r(rows, 16).cuda(), tokens=torch.arange(n).remainder(rows).cuda(),
                 gfeatures=r(n, 16).cuda(), gmatrix=r(64, 64).cuda(),
                 **{k: v.cuda() for k, v in cpu.items()})
    exec(_step(), space)   # noqa: S102
    F = torch.nn.functional
    d = {k: v.double().requires_grad_(k != "gout") for k, v in cpu.items()}
    y = F.silu(F.group_norm(d["image"].view(1, H * W, 16).transpose(1, 2), 4, d["gamma"], d["beta"],
                            1e-5).transpose(1, 2))
    out = F.linear(F.silu(F.linear(y, d["weight"], d["bias"])), d["weight2"], d["bias2"]) + y
    keep = (ref.dropout_words(out.numel(), 77, 5) >= round(0.1 * 2 ** 32)).view(out.shape)
    out = torch.where(keep, out / 0.9, 0.0)
    names = {"gx": "image", "ggamma": "gamma", "gbeta": "beta", "gweight": "weight", "gbias": "bias",
             "gweight2": "weight2", "gbias2": "bias2"}
    want = dict(zip(names, torch.autograd.grad(out, [d[k] for k in names.values()],
                                               d["gout"].view(out.shape))))
    # each of some four products and sums of 600 rows within 1e-6 of its norm
    close = lambda a, b: float((a.cpu().double().reshape(b.shape) - b).norm() / b.norm()) <= 1e-5  # noqa: E731
    assert close(space["out"], out.detach())
    for k, v in want.items():
        assert close(space[k], v), k
    space["ops"].close()
