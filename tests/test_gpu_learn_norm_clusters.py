"""Group norm of small images whose pixels end inside a warp: the threads of a
warp part ways before the barriers of the cluster that shares the image."""
from __future__ import annotations

import pytest
import torch

import learn_reference as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=1 << 26)
    yield o
    assert o.status() == 0
    o.close()


# a block has 256 threads; so many along the channels of so many pixels: 5 x 51, 7 x 36, 75 x 3,
# 3 x 85 (channels one by one), 100 x 2, 255 x 1; over one, two, four and eight blocks
CHANNELS = [(20, 4), (28, 7), (300, 3), (3, 1), (100, 25), (255, 5)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("channels", CHANNELS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("pixels", [1, 2, 5, 13, 37, 61])
def test_pixels_that_end_inside_a_warp(ops, channels, pixels, dtype):
    C, G = channels
    gen = torch.Generator().manual_seed(C + pixels)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, dy = r(3, pixels, C).to(TYPES[dtype]), r(3, pixels, C).to(TYPES[dtype])
    w, b = 1 + 0.3 * r(C), 0.3 * r(C)
    args = x.cuda(), G, w.cuda(), b.cuda(), 1e-5, "silu"
    y, stats = ops.group_norm(*args)
    want, s_want, e_y, e_s = ref.group_norm(x, G, w, b, 1e-5, "silu")
    assert not ref.outside(stats, s_want, e_s).any() and not ref.outside(y, want, e_y).any()
    back = dy.cuda(), x.cuda(), stats, G, w.cuda(), b.cuda(), "silu"
    got = ops.group_norm_backward(*back)
    want, bounds = ref.group_norm_backward(dy, x, stats.cpu(), G, w, b, "silu")
    for g, v, e in zip(got, want, bounds):
        assert not ref.outside(g, v, e).any()
    for _ in range(3):
        assert all(map(torch.equal, (y, stats), ops.group_norm(*args)))
        assert all(map(torch.equal, got, ops.group_norm_backward(*back)))
