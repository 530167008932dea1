"""Channels-last group norm with an activation, forward and backward, against
its definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

import learn_reference as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=1 << 28)
    yield o
    assert o.status() == 0
    o.close()


def _inputs(N, P, C, T, seed, shift=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (r(N, P, C) * (0.5 + torch.rand(C, generator=gen)) + shift * r(C)).to(T)
    return x, r(N, P, C).to(T), 1 + 0.3 * r(C), 0.3 * r(C)


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _inside(got, want, bound, what):
    bad = ref.outside(got, want, bound)
    e = ((got.cpu().double() - want).abs() / (bound + 1e-30)).max()
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {float(e)} of the bound"


CASES = [
    # images, pixels, channels, groups
    (1, 1, 1, 1), (2, 1, 8, 2), (1, 2, 3, 3), (3, 17, 6, 2), (1, 960, 16, 4), (2, 333, 20, 4),
    (1, 5000, 16, 1), (1, 5000, 16, 16), (2, 700, 64, 8), (1, 129, 320, 32), (1, 40, 2048, 32),
    (1, 9, 4096, 1), (2, 11, 1030, 2), (5, 64, 24, 3), (1, 4097, 5, 5), (1, 300, 1500, 4),
]


@pytest.mark.parametrize("name", ["none", "silu", "relu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_group_norm(ops, case, dtype, name):
    N, P, C, G = case
    x, dy, w, b = _inputs(N, P, C, TYPES[dtype], 100 + P + C)
    if name == "none":
        w = b = None
    xc, dyc, wc, bc = _cuda(x, dy, w, b)
    y, stats = ops.group_norm(xc, G, wc, bc, 1e-5, name)
    want, s_want, e_y, e_s = ref.group_norm(x, G, w, b, 1e-5, name)
    _inside(stats, s_want, e_s, "stats")
    _inside(y, want, e_y, "y")
    assert y.dtype == x.dtype
    got = ops.group_norm_backward(dyc, xc, stats, G, wc, bc, name)
    want, bounds = ref.group_norm_backward(dy, x, stats.cpu(), G, w, b, name)
    for g, v, e, what in zip(got, want, bounds, ("dx", "dw", "db")):
        _inside(g, v, e, what)


@pytest.mark.parametrize("name", ["none", "silu"])
def test_gradient_is_the_derivative(ops, name):
    """Central differences of <dy, y> in 64 bits, in random directions of x,
    the weights and the biases; step h: an error of order h^2 of the third
    derivative (below 1e-6 of the scale here) and eps / h of the rounding."""
    N, P, C, G = 2, 50, 12, 3
    x, dy, w, b = _inputs(N, P, C, torch.float32, 7)
    xc, dyc, wc, bc = _cuda(x, dy, w, b)
    _, stats = ops.group_norm(xc, G, wc, bc, 1e-5, name)
    got = ops.group_norm_backward(dyc, xc, stats, G, wc, bc, name)
    gen = torch.Generator().manual_seed(8)
    h = 1e-4
    for k, t in enumerate((x, w, b)):
        d = torch.randn(t.shape, generator=gen).double()

        def loss(s):
            args = [x.double(), w.double(), b.double()]
            args[k] = args[k] + s * d
            return (dy.double() * ref.group_norm(args[0], G, args[1], args[2], 1e-5, name)[0]).sum()

        numeric = (loss(h) - loss(-h)) / (2 * h)
        analytic = (got[k].cpu().double() * d).sum()
        scale = (got[k].cpu().double() * d).abs().sum()
        assert abs(numeric - analytic) <= 2e-5 * scale


def test_mean_far_above_the_spread_and_an_outlier(ops):
    """The second moment does not cancel: a mean of 1000 standard deviations,
    and a first pixel far from all others."""
    gen = torch.Generator().manual_seed(21)
    x = torch.randn(2, 3000, 16, generator=gen) + 1000.0
    x[1, 0] = -5000.0
    y, stats = ops.group_norm(x.cuda(), 4, act="silu")
    want, s_want, e_y, e_s = ref.group_norm(x, 4, None, None, 1e-5, "silu")
    _inside(stats, s_want, e_s, "stats")
    _inside(y, want, e_y, "y")


def test_constant_image(ops):
    """No variance: y = act(bias), the gradient of x finite."""
    x = torch.full((1, 100, 8), 3.0).cuda()
    b = torch.linspace(-1, 1, 8).cuda()
    y, stats = ops.group_norm(x, 2, None, b, 1e-5, "relu")
    assert torch.equal(y, torch.relu(b).expand(1, 100, 8))
    assert stats[..., 0].eq(3.0).all()
    dx, _, db = ops.group_norm_backward(torch.ones_like(x), x, stats, 2, None, b, "relu")
    assert dx.isfinite().all() and torch.equal(db, 100.0 * (b > 0))


def test_nan_stays_in_its_group(ops):
    x = torch.randn(2, 50, 8, generator=torch.Generator().manual_seed(3)).cuda()
    x[0, 7, 2] = float("nan")
    y, stats = ops.group_norm(x, 2, act="silu")
    assert y[0, :, :4].isnan().all() and not y[0, :, 4:].isnan().any()
    assert not y[1].isnan().any() and stats[0, 0].isnan().all()


def test_nothing_to_do(ops):
    for shape in ((0, 5, 8), (2, 0, 8)):
        x = torch.empty(shape, device="cuda")
        y, stats = ops.group_norm(x, 4, eps=0.25)
        assert y.shape == x.shape and stats.shape == (shape[0], 4, 2)
        assert stats[..., 0].eq(0).all() and stats[..., 1].eq(2).all()
        dx, dw, db = ops.group_norm_backward(x, x, stats, 4)
        assert dw.eq(0).all() and db.eq(0).all()


def test_only_what_is_wanted_and_in_place(ops):
    x, dy, w, b = _inputs(2, 400, 16, torch.float32, 31)
    x, dy, w, b = _cuda(x, dy, w, b)
    y, stats = ops.group_norm(x, 4, w, b, act="silu")
    full = ops.group_norm_backward(dy, x, stats, 4, w, b, "silu")
    for k, name in enumerate(("x", "weight", "bias")):
        part = ops.group_norm_backward(dy, x, stats, 4, w, b, "silu", want=(name,))
        assert [p is not None for p in part] == [j == k for j in range(3)]
        assert torch.equal(part[k], full[k])
    g = dy.clone()
    ops.group_norm_backward(g, x, stats, 4, w, b, "silu", grad_x=g)
    assert torch.equal(g, full[0])
    z = x.clone()
    ops.group_norm(z, 4, w, b, act="silu", out=z)
    assert torch.equal(z, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_images_at_any_element_alignment(ops, dtype):
    T = TYPES[dtype]
    x, dy, w, b = _inputs(1, 210, 16, T, 41)

    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=T, device="cuda")
        flat[1:] = t.reshape(-1).cuda()
        return flat[1:].view(t.shape)

    wc, bc = _cuda(w, b)
    y, stats = ops.group_norm(off(x), 4, wc, bc, act="silu")
    want, s_want, e_y, e_s = ref.group_norm(x, 4, w, b, 1e-5, "silu")
    _inside(y, want, e_y, "y")
    got = ops.group_norm_backward(off(dy), off(x), stats, 4, wc, bc, "silu")
    want, bounds = ref.group_norm_backward(dy, x, stats.cpu(), 4, w, b, "silu")
    for g, v, e, what in zip(got, want, bounds, ("dx", "dw", "db")):
        _inside(g, v, e, what)


def test_same_bits_every_time_and_on_another_stream(ops):
    x, dy, w, b = _cuda(*_inputs(3, 20_000, 16, torch.float32, 51))
    y, stats = ops.group_norm(x, 4, w, b, act="silu")
    want = ops.group_norm_backward(dy, x, stats, 4, w, b, "silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, stats2 = ops.group_norm(x, 4, w, b, act="silu")
        got = ops.group_norm_backward(dy, x, stats2, 4, w, b, "silu")
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(stats, stats2)
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_refusals(ops):
    from splat_rendering_gb300 import pulsar as pl
    x = torch.zeros(1, 10, 12, device="cuda")
    with pytest.raises(pl.PulsarError):
        ops.group_norm(x, 5)
    with pytest.raises(pl.PulsarError):
        ops.group_norm(x, 4, eps=-1.0)
    with pytest.raises(pl.PulsarError):
        ops.group_norm(torch.zeros(1, 2, 4100, device="cuda"), 4)
    with pytest.raises(ValueError, match="act"):
        ops.group_norm(x, 4, act="gelu")
    with pytest.raises(ValueError, match="not contiguous"):
        ops.group_norm(x.transpose(1, 2), 5)
    with pytest.raises(ValueError, match="shape"):
        ops.group_norm(x, 4, torch.ones(11, device="cuda"))
    with pytest.raises(TypeError):
        ops.group_norm(x, 4, torch.ones(12, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        ops.group_norm(x.half(), 4)
    _, stats = ops.group_norm(x, 4)
    with pytest.raises(TypeError):
        ops.group_norm_backward(x.bfloat16(), x, stats, 4)
    with pytest.raises(ValueError, match="shape"):
        ops.group_norm_backward(x, x, stats, 3)
