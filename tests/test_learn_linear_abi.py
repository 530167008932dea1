"""Host-side checks of the linear layer's and dropout's entry points (no GPU needed)."""
from __future__ import annotations

import pytest
import torch

import linear_reference as ref


@pytest.fixture(scope="module")
def lib():
    from splat_rendering_gb300 import build, pulsar
    build.build()
    return pulsar.load()


def test_null_handles(lib):
    from splat_rendering_gb300 import pulsar as pl
    assert lib.pulsar_linear_forward(None, None, None, 0, 1, 1, None, None, 0, 0, None, None,
                                     None) == pl.ERR_ARG
    assert lib.pulsar_linear_backward(None, None, None, None, None, 0, 1, 1, 0, 0, None, None, None,
                                      None) == pl.ERR_ARG
    assert lib.pulsar_dropout(None, None, None, 0, 0.5, 0, 0, None, 0, None, None) == pl.ERR_ARG


def test_workspace_sizes(lib):
    from splat_rendering_gb300 import pulsar as pl
    assert pl.linear_workspace(0, 1, 1, torch.float32) >= 0
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 65537, 1), (1, 1, 65537), (0x7fff0001, 1, 1),
                ((1 << 22) + 1, 65536, 1), ((1 << 22) + 1, 1, 65536)):
        with pytest.raises(pl.PulsarError):
            pl.linear_workspace(*bad, torch.float32)
    with pytest.raises(TypeError):
        pl.linear_workspace(4, 4, 4, torch.float16)


@pytest.fixture
def ops(monkeypatch):
    """A Learner whose tensors may lie on the host and whose library is not reached."""
    from splat_rendering_gb300 import pulsar as pl
    o = object.__new__(pl.Learner)
    o.handle, o.device, o._torch, o._dev = 0, -1, torch, "cpu"
    monkeypatch.setattr(pl.Learner, "_stream", lambda self, s: 0)

    class Library:
        def __getattr__(self, name):
            def reached(*args):
                raise AssertionError(f"the call reached the library ({name})")
            return reached

    o._lib = Library()
    return o


def test_refused_before_the_library(ops):
    x, w = torch.zeros(2, 5, 8), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="weight"):
        ops.linear(x, w[0])
    with pytest.raises(ValueError, match="x has shape"):
        ops.linear(x, torch.zeros(4, 7))
    with pytest.raises(ValueError, match="act"):
        ops.linear(x, w, act="gelu")
    with pytest.raises(TypeError):
        ops.linear(x.half(), w.half())
    with pytest.raises(TypeError, match="weight"):
        ops.linear(x, w.bfloat16())
    with pytest.raises(TypeError, match="bias"):
        ops.linear(x, w, torch.zeros(4).bfloat16())
    with pytest.raises(ValueError, match="bias"):
        ops.linear(x, w, torch.zeros(8))
    with pytest.raises(ValueError, match="residual"):
        ops.linear(x, w, None, x)
    with pytest.raises(ValueError, match="contiguous"):
        ops.linear(x.transpose(0, 1), w)
    with pytest.raises(ValueError, match="contiguous"):
        ops.linear(x, torch.zeros(8, 4).T)
    with pytest.raises(ValueError, match="pre is needed"):
        ops.linear_backward(torch.zeros(2, 5, 4), x, w, act="silu")
    with pytest.raises(ValueError, match="grad_y"):
        ops.linear_backward(x, x, w)
    with pytest.raises(ValueError, match="pre"):
        ops.linear_backward(torch.zeros(2, 5, 4), x, w, x, act="relu")
    for seed, offset in ((-1, 0), (1 << 64, 0), (0, -1), (0, 1 << 63)):
        with pytest.raises(ValueError, match="seed"):
            ops.dropout(x, 0.5, seed, offset)
    with pytest.raises(ValueError, match="counter"):
        ops.dropout(x, 0.5, 0, counter=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError, match="counter"):
        ops.dropout(x, 0.5, 0, counter=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="residual"):
        ops.dropout(x, 0.5, 0, residual=x[0])


def test_reference_forms_agree_with_torch():
    """The tests' 64-bit forms against torch's own operators and its autograd."""
    gen = torch.Generator().manual_seed(1)
    F = torch.nn.functional
    x = torch.randn(3, 7, 12, generator=gen).double().requires_grad_()
    w = torch.randn(5, 12, generator=gen).double().requires_grad_()
    b = torch.randn(5, generator=gen).double().requires_grad_()
    r, dy = (torch.randn(3, 7, 5, generator=gen).double() for _ in range(2))
    for name, f in (("none", lambda v: v), ("silu", F.silu), ("relu", F.relu)):
        z = F.linear(x, w, b)
        want = torch.autograd.grad(f(z) + r, (x, w, b), dy, retain_graph=True)
        (y, zz), _ = ref.linear(x.detach(), w.detach(), b.detach(), r, name)
        assert torch.allclose(y, (f(z) + r).detach(), rtol=1e-12, atol=1e-12)
        grads, _ = ref.linear_backward(dy, x.detach(), w.detach(), zz, name)
        for g, v in zip(grads, want):
            assert torch.allclose(g, v, rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("rounds,ctr,key,want", [
    (7, (0, 0, 0, 0), (0, 0), (0x5f6fb709, 0x0d893f64, 0x4f121f81, 0x4f730a48)),
    (10, (0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    (10, (0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
])
def test_philox_known_answers(rounds, ctr, key, want):
    """The published known answers of the generator."""
    assert tuple(ref.philox(torch.tensor(ctr), key, rounds).tolist()) == want
