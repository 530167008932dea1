"""The linear layer with bias, activation and residual, and its gradients,
against their definitions in 64 bits."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ops():
    from splat_rendering_gb300 import pulsar as pl
    o = pl.Learner(workspace_bytes=1 << 29)
    yield o
    assert o.status() == 0
    o.close()


def _inputs(M, K, N, T, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return ((scale * r(M, K)).to(T), (r(N, K) / K ** 0.5).to(T), 0.3 * r(N), r(M, N).to(T),
            (1e-2 * r(M, N)).to(T))


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _inside(got, want, bound, what):
    bad = ref.outside(got, want, bound)
    e = ((got.cpu().double() - want).abs() / (bound + 1e-30)).max()
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {float(e)} of the bound"


def _near(got, want, what):
    """In 32 bits also as near, in all, as sums in 32 bits are."""
    if got.dtype == torch.float32 and float(want.norm()) > 0:
        e = float((got.cpu().double() - want).norm() / want.norm())
        assert e <= 1e-6, f"{what}: {e} of its norm"


# rows, inputs, outputs: one row and few, one input, one output, whole tiles, ragged ones, a
# contraction in parts, several column blocks
CASES = [
    (1, 1, 1), (1, 4096, 300), (2, 19, 64), (3, 17, 5), (4, 1000, 33), (5, 16, 64), (17, 64, 3),
    (128, 64, 128), (129, 65, 127), (960, 16, 64), (1000, 19, 64), (200, 1, 300), (257, 200, 300),
    (300, 509, 700), (130, 4096, 130), (16, 2048, 4096), (5001, 64, 64), (9000, 3, 3),
    (2000, 128, 128), (700, 256, 512), (1111, 100, 72), (20_000, 24, 40),
]


@pytest.mark.parametrize("name", ["none", "silu", "relu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_linear(ops, case, dtype, name):
    M, K, N = case
    x, w, b, r, dy = _inputs(M, K, N, TYPES[dtype], 100 + M + K + N)
    if name == "none":
        b = None
    if name == "relu":
        r = None
    xc, wc, bc, rc, dyc = _cuda(x, w, b, r, dy)
    y, z = ops.linear(xc, wc, bc, rc, name, want_pre=True)
    (y_want, z_want), (e_y, e_z) = ref.linear(x, w, b, r, name)
    _inside(z, z_want, e_z, "z")
    _inside(y, y_want, e_y, "y")
    _near(z, z_want, "z")
    assert y.dtype == x.dtype
    y2, none = ops.linear(xc, wc, bc, rc, name)
    assert none is None and torch.equal(y, y2)
    got = ops.linear_backward(dyc, xc, wc, z, name)
    want, bounds = ref.linear_backward(dy, x, w, z.cpu(), name)
    for g, v, e, what in zip(got, want, bounds, ("dx", "dw", "db")):
        _inside(g, v, e, what)
        _near(g, v, what)


@pytest.mark.parametrize("name", ["none", "silu"])
def test_gradient_is_the_derivative(ops, name):
    """Central differences of <dy, y> in 64 bits, in random directions of x, the weight and the
    bias; step h: an error of order h^2 of the third derivative and eps / h of the rounding."""
    x, w, b, _, dy = _inputs(60, 40, 24, torch.float32, 7)
    xc, wc, bc, dyc = _cuda(x, w, b, dy)
    _, z = ops.linear(xc, wc, bc, act=name, want_pre=True)
    got = ops.linear_backward(dyc, xc, wc, z, name)
    gen = torch.Generator().manual_seed(8)
    h = 1e-4
    for k, t in enumerate((x, w, b)):
        d = torch.randn(t.shape, generator=gen).double()

        def loss(s):
            args = [x.double(), w.double(), b.double()]
            args[k] = args[k] + s * d
            return (dy.double() * ref.linear(*args, None, name)[0][0]).sum()

        numeric = (loss(h) - loss(-h)) / (2 * h)
        analytic = (got[k].cpu().double() * d).sum()
        scale = (got[k].cpu().double() * d).abs().sum()
        assert abs(numeric - analytic) <= 2e-5 * scale


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(3, 64, 64), (300, 64, 64), (500, 136, 72)],
                         ids=lambda c: "-".join(map(str, c)))
def test_any_element_alignment(ops, case, dtype):
    T = TYPES[dtype]
    x, w, b, r, dy = _inputs(*case, T, 41)

    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.reshape(-1).cuda()
        return flat[1:].view(t.shape)

    new = lambda t: off(torch.zeros_like(t))  # noqa: E731
    y, z = ops.linear(off(x), off(w), off(b), off(r), "silu", out=new(r), pre=new(r))
    (y_want, z_want), (e_y, e_z) = ref.linear(x, w, b, r, "silu")
    _inside(z, z_want, e_z, "z")
    _inside(y, y_want, e_y, "y")
    got = ops.linear_backward(off(dy), off(x), off(w), z, "silu", grad_x=new(x), grad_weight=new(w),
                              grad_bias=new(b))
    want, bounds = ref.linear_backward(dy, x, w, z.cpu(), "silu")
    for g, v, e, what in zip(got, want, bounds, ("dx", "dw", "db")):
        _inside(g, v, e, what)


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e15, 1e30])
def test_float32_range(ops, scale):
    """No scales: rows of every magnitude keep their own relative accuracy (down to where the
    products' last parts leave float32's range)."""
    x, w, b, _, dy = _inputs(300, 200, 90, torch.float32, 51)
    x[::2] *= scale
    xc, wc = _cuda(x, w)
    y, _ = ops.linear(xc, wc)
    (want, _), (e, _) = ref.linear(x, w, None, None, "none")
    _inside(y, want, e, "y")
    for rows in (slice(0, None, 2), slice(1, None, 2)):
        _near(y[rows], want[rows], "y")


def test_non_finite_rows_stay_alone(ops):
    for T in TYPES.values():
        for M in (3, 300):
            x, w, b, r, dy = _inputs(M, 70, 50, T, 61)
            x[1, 3], x[2, 5] = float("inf"), float("nan")
            w[7, 2] = float("-inf")
            y, _ = ops.linear(*_cuda(x, w, b))
            bad = ~y.isfinite().cpu()
            assert bad[1].all() and bad[2].all() and bad[:, 7].all()
            bad[1], bad[2], bad[:, 7] = False, False, False
            assert not bad.any()


def test_nothing_to_do(ops):
    x, w = torch.empty(0, 8, device="cuda"), torch.ones(5, 8, device="cuda")
    y, z = ops.linear(x, w, want_pre=True)
    assert y.shape == z.shape == (0, 5)
    dx, dw, db = ops.linear_backward(y, x, w, z, "silu")
    assert dx.shape == (0, 8) and dw.eq(0).all() and db.eq(0).all()


def test_leading_dimensions_and_a_vector(ops):
    x, w, b, r, _ = _cuda(*_inputs(60, 24, 40, torch.float32, 71))
    y, z = ops.linear(x, w, b, r, "silu", want_pre=True)
    y3, z3 = ops.linear(x.view(3, 4, 5, 24), w, b, r.view(3, 4, 5, 40), "silu", want_pre=True)
    assert y3.shape == (3, 4, 5, 40) and torch.equal(y3.view(60, 40), y)
    assert torch.equal(z3.view(60, 40), z)
    y1, _ = ops.linear(x[0], w, b)
    assert y1.shape == (40,)


def test_only_what_is_wanted_and_in_place(ops):
    for T in TYPES.values():
        x, w, b, r, dy = _cuda(*_inputs(400, 48, 80, T, 81))
        y, z = ops.linear(x, w, b, r, "silu", want_pre=True)
        full = ops.linear_backward(dy, x, w, z, "silu")
        for k, name in enumerate(("x", "weight", "bias")):
            part = ops.linear_backward(dy, x, w, z, "silu", want=(name,))
            assert [p is not None for p in part] == [j == k for j in range(3)]
            assert torch.equal(part[k], full[k])
        assert ops.linear_backward(dy, x, w, z, "silu", want=()) == (None, None, None)
        ops.linear(x, w, b, r, "silu", out=r)
        assert torch.equal(r, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_every_time_and_on_another_stream(ops, dtype):
    x, w, b, r, dy = _cuda(*_inputs(30_000, 64, 64, TYPES[dtype], 91))

    def work():
        y, z = ops.linear(x, w, b, r, "silu", want_pre=True)
        return [y, z, *ops.linear_backward(dy, x, w, z, "silu")]

    want = work()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = work()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_the_workspace_is_enough():
    """The same bits as with room to spare, and nothing less is taken."""
    from splat_rendering_gb300 import pulsar as pl
    for T in TYPES.values():
        for M, K, N in ((300, 70, 50), (40, 4096, 200), (20_000, 64, 64)):
            x, w, b, r, dy = _cuda(*_inputs(M, K, N, T, 95))
            need = pl.linear_workspace(M, K, N, T)
            outs = []
            for room in (need, need + (1 << 26)):
                o = pl.Learner(workspace_bytes=room)
                y, z = o.linear(x, w, b, r, "silu", want_pre=True)
                outs.append([y, z, *o.linear_backward(dy, x, w, z, "silu")])
                o.status()
                o.close()
            assert all(torch.equal(p, q) for p, q in zip(*outs))
            o = pl.Learner(workspace_bytes=need - 1)
            with pytest.raises(pl.PulsarError, match="workspace"):
                o.linear(x, w)
            with pytest.raises(pl.PulsarError, match="workspace"):
                o.linear_backward(dy, x, w)
            o.close()


def test_refusals(ops):
    from splat_rendering_gb300 import pulsar as pl
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(5, 8, device="cuda")
    with pytest.raises(ValueError, match="not on"):
        ops.linear(x.cpu(), w)
    with pytest.raises(ValueError, match="not on"):
        ops.linear(x, w, torch.zeros(5))
    with pytest.raises(ValueError, match="contiguous"):
        ops.linear(x[:, ::2], w[:, :4].contiguous())
    with pytest.raises(pl.PulsarError):
        ops.linear(x, torch.zeros(65537, 8, device="cuda"))
