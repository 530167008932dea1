"""Codebook embedding and its gradient against their definitions in 64 bits."""
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


def _tokens(kind, n, rows, gen, index):
    if kind == "uniform":
        t = torch.randint(0, rows, (n,), generator=gen)
    elif kind == "one":            # every token names the same row
        t = torch.full((n,), rows // 2)
    elif kind == "masked":         # no token names a row
        t = torch.full((n,), -1)
    elif kind == "sorted":
        t = torch.sort(torch.randint(0, rows, (n,), generator=gen)).values
    else:                          # few popular rows, many masked
        t = (torch.rand(n, generator=gen) ** 4 * rows).long().clamp(max=rows - 1)
        t[torch.rand(n, generator=gen) < 0.3] = -7
    return t.to(torch.int32 if index == "i32" else torch.int64)


CASES = [
    # n, rows, dim, tokens
    (1, 1, 1, "uniform"), (0, 5, 4, "uniform"), (1, 300, 16, "masked"), (33, 7, 3, "uniform"),
    (1000, 256, 3, "mixed"), (1000, 1, 16, "uniform"), (4099, 65536, 4, "uniform"),
    (2049, 255, 5, "one"), (2500, 256, 8, "sorted"), (5000, 3, 64, "mixed"),
    (70001, 8192, 16, "mixed"), (70001, 70000, 1, "mixed"), (65537, 40, 16, "one"),
    (1500, 100, 1024, "mixed"), (777, 50, 1030, "mixed"), (300, 17, 4100, "uniform"),
    (20000, 1 << 20, 2, "uniform"), (3000, 513, 24, "masked"),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("index", ["i32", "i64"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_embedding_and_gradient(ops, case, index, dtype):
    n, rows, dim, kind = case
    gen = torch.Generator().manual_seed(n * 7 + rows + dim)
    table = torch.randn(rows, dim, generator=gen).to(TYPES[dtype])
    tokens = _tokens(kind, n, rows, gen, index)
    grad = torch.randn(n, dim, generator=gen).to(TYPES[dtype])
    scale = 1.7
    out = ops.embed(table.cuda(), tokens.cuda(), scale).cpu()
    want = ref.embed(table, tokens, float(torch.tensor(scale, dtype=torch.float32)))
    assert out.shape == (n, dim) and out.dtype == TYPES[dtype]
    assert not ref.outside(out, want, ref.U32 * want.abs()).any()
    # the gradient overwrites whatever its output held
    got = torch.full((rows, dim), float("nan"), dtype=TYPES[dtype], device="cuda")
    ops.embed_backward(grad.cuda(), tokens.cuda(), rows, scale, grad_table=got)
    want, bound = ref.embed_backward(grad, tokens, rows,
                                     float(torch.tensor(scale, dtype=torch.float32)))
    assert not ref.outside(got, want, bound).any()


def test_gradient_is_the_derivative(ops):
    """<dout, out(table + d) - out(table)> = <dtable, d>: the embedding is linear."""
    gen = torch.Generator().manual_seed(5)
    table, d = (torch.randn(90, 12, generator=gen) for _ in range(2))
    tokens = torch.randint(-3, 90, (7, 600), generator=gen)
    grad = torch.randn(7, 600, 12, generator=gen)
    dt = ops.embed_backward(grad.cuda(), tokens.cuda(), 90, 0.5).cpu().double()
    diff = ref.embed(table.double() + d.double(), tokens, 0.5) - ref.embed(table, tokens, 0.5)
    lhs, rhs = (grad.double() * diff).sum(), (dt * d.double()).sum()
    _, bound = ref.embed_backward(grad, tokens, 90, 0.5)
    assert abs(lhs - rhs) <= (bound * d.abs().double()).sum() + 1e-9


def test_same_bits_every_time(ops):
    gen = torch.Generator().manual_seed(9)
    tokens = _tokens("mixed", 50_000, 1000, gen, "i32").cuda()
    grad = torch.randn(50_000, 16, generator=gen).cuda()
    first = ops.embed_backward(grad, tokens, 1000)
    for _ in range(3):
        ops.embed_backward(grad[:777].contiguous(), tokens[:777].contiguous(), 1000)
        assert torch.equal(first, ops.embed_backward(grad, tokens, 1000))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_at_any_element_alignment(ops, dtype):
    """Tensors that begin off a 16-byte boundary take the element path: same values."""
    gen = torch.Generator().manual_seed(11)
    T = TYPES[dtype]
    table, grad = torch.randn(64, 16, generator=gen).to(T), torch.randn(900, 16, generator=gen).to(T)
    tokens = torch.randint(0, 64, (900,), generator=gen).cuda()

    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=T, device="cuda")
        flat[1:] = t.reshape(-1).cuda()
        return flat[1:].view(t.shape)

    assert torch.equal(ops.embed(off(table), tokens), ops.embed(table.cuda(), tokens))
    a, b = ops.embed_backward(off(grad), tokens, 64), ops.embed_backward(grad.cuda(), tokens, 64)
    want, bound = ref.embed_backward(grad, tokens.cpu(), 64, 1.0)
    for g in (a, b):
        assert not ref.outside(g, want, bound).any()


def test_masked_rows_stay_zero_and_infinities_pass(ops):
    table = torch.tensor([[1.0, float("inf")], [float("nan"), 2.0]], device="cuda")
    tokens = torch.tensor([-1, 0, 1], device="cuda")
    out = ops.embed(table, tokens, 3.0).cpu()
    assert out[0].tolist() == [0.0, 0.0] and out[1].tolist() == [3.0, float("inf")]
    assert out[2].isnan().tolist() == [True, False]
    # a NaN in the gradient of a masked token goes nowhere
    g = torch.tensor([[float("nan"), float("inf")], [1.0, 2.0], [3.0, 4.0]], device="cuda")
    assert ops.embed_backward(g, tokens, 2).cpu().tolist() == [[1.0, 2.0], [3.0, 4.0]]


def test_token_outside_the_table_is_reported(ops):
    from splat_rendering_gb300 import pulsar as pl
    table = torch.ones(4, 4, device="cuda")
    tokens = torch.tensor([0, 4, 3, 1 << 40], device="cuda")
    out = ops.embed(table, tokens)
    with pytest.raises(pl.PulsarError, match="outside the table"):
        ops.status()
    assert out.cpu()[:, 0].tolist() == [1.0, 0.0, 1.0, 0.0]
    g = ops.embed_backward(torch.ones(4, 4, device="cuda"), tokens, 4)
    assert ops.status(raise_on_error=False) == pl.ERR_INDEX
    assert ops.status(raise_on_error=False) == pl.OK
    assert g.cpu()[:, 0].tolist() == [1.0, 0.0, 0.0, 1.0]


def test_on_another_stream(ops):
    gen = torch.Generator().manual_seed(13)
    grad = torch.randn(30_000, 8, generator=gen).cuda()
    tokens = torch.randint(0, 500, (30_000,), generator=gen).cuda()
    want = ops.embed_backward(grad, tokens, 500)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        inside = ops.embed_backward(grad, tokens, 500)
    given = torch.empty_like(want)
    ops.embed_backward(grad, tokens, 500, grad_table=given, stream=s)
    s.synchronize()
    assert torch.equal(inside, want) and torch.equal(given, want)


def test_refusals(ops):
    from splat_rendering_gb300 import pulsar as pl
    table = torch.ones(8, 8, device="cuda")
    tokens = torch.zeros(5, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="not contiguous"):
        ops.embed(table.t(), tokens)
    with pytest.raises(ValueError, match="not on cuda"):
        ops.embed(table.cpu(), tokens)
    with pytest.raises(TypeError):
        ops.embed(table.double(), tokens)
    with pytest.raises(TypeError):
        ops.embed(table, tokens.float())
    with pytest.raises(ValueError, match="shape"):
        ops.embed(table, tokens, out=torch.empty(4, 8, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        ops.embed_backward(torch.ones(4, 8, device="cuda"), tokens, 8)
    with pytest.raises(pl.PulsarError):
        ops.embed(table, tokens, scale=float("inf"))
    with pytest.raises(pl.PulsarError):
        ops.embed_backward(torch.ones(5, 8, device="cuda"), tokens, 0)
    small = pl.Learner(workspace_bytes=16)
    with pytest.raises(pl.PulsarError, match="workspace"):
        small.embed_backward(torch.ones(5, 8, device="cuda"), tokens, 8)
    small.close()
