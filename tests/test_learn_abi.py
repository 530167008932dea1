"""Host-side checks of the learned parts' entry points (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import learn_reference as ref


@pytest.fixture(scope="module")
def lib():
    from splat_rendering_gb300 import build, pulsar
    build.build()
    return pulsar.load()


def test_null_handles_and_bad_limits(lib):
    from splat_rendering_gb300 import pulsar as pl
    h = ctypes.c_void_p()
    assert lib.pulsar_learn_create(None, 0, 0) == pl.ERR_ARG
    assert lib.pulsar_learn_create(ctypes.byref(h), 0, -1) == pl.ERR_ARG
    assert lib.pulsar_learn_destroy(None) == pl.ERR_ARG
    assert lib.pulsar_learn_status(None, None) == pl.ERR_ARG
    assert lib.pulsar_embed_forward(None, None, None, 0, 1, 1, 1.0, 0, 0, None, None) == pl.ERR_ARG
    assert lib.pulsar_embed_backward(None, None, None, 0, 1, 1, 1.0, 0, 0, None, None) == pl.ERR_ARG
    assert lib.pulsar_group_norm_forward(None, None, 0, 0, 1, 1, None, None, 1e-5, 0, 0, None, None,
                                         None) == pl.ERR_ARG
    assert lib.pulsar_group_norm_backward(None, None, None, None, 0, 0, 1, 1, None, None, 0, 0,
                                          None, None, None, None) == pl.ERR_ARG
    assert lib.pulsar_orthogonalize(None, None, 0, 1, 1, 5, None, 1e-7, 0, None, None) == pl.ERR_ARG
    assert "workspace" in pl.strerror(pl.ERR_WORKSPACE)
    assert "table" in pl.strerror(pl.ERR_INDEX)


def test_workspace_sizes(lib):
    from splat_rendering_gb300 import pulsar as pl
    assert pl.embed_workspace(0, 1, 1) == 0
    assert pl.embed_workspace(1000, 256, 3) >= 4 * 4 * 1000
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 65537), (0x7fff0001, 1, 1)):
        with pytest.raises(pl.PulsarError):
            pl.embed_workspace(*bad)
    assert pl.group_norm_workspace(0, 10, 8, 4) == 0
    for bad in ((-1, 1, 8, 4), (1, -1, 8, 4), (1, 1, 8, 3), (1, 1, 8, 0), (1, 1, 4100, 4),
                (65536, 1, 8, 4)):
        with pytest.raises(pl.PulsarError):
            pl.group_norm_workspace(*bad)
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, 65537), (65536, 1, 1)):
        with pytest.raises(pl.PulsarError):
            pl.orthogonalize_workspace(*bad, torch.float32)
    with pytest.raises(TypeError):
        pl.orthogonalize_workspace(1, 4, 4, torch.float16)


def test_reference_forms_agree_with_torch():
    """The tests' 64-bit forms against torch's own operators and its autograd."""
    gen = torch.Generator().manual_seed(1)
    F = torch.nn.functional
    x = torch.randn(2, 30, 12, generator=gen).double().requires_grad_()
    w, b = (torch.randn(12, generator=gen).double().requires_grad_() for _ in range(2))
    dy = torch.randn(2, 30, 12, generator=gen).double()
    y = F.silu(F.group_norm(x.transpose(1, 2), 3, w, b, 1e-5)).transpose(1, 2)
    want = torch.autograd.grad(y, (x, w, b), dy)
    got, stats, _, _ = ref.group_norm(x.detach(), 3, w.detach(), b.detach(), 1e-5, "silu")
    assert torch.allclose(got, y.detach(), rtol=1e-12, atol=1e-12)
    grads, _ = ref.group_norm_backward(dy, x.detach(), stats, 3, w.detach(), b.detach(), "silu")
    for g, v in zip(grads, want):
        assert torch.allclose(g, v, rtol=1e-10, atol=1e-10)
    table = torch.randn(9, 4, generator=gen).double().requires_grad_()
    tokens = torch.randint(0, 9, (50,), generator=gen)
    d = torch.randn(50, 4, generator=gen).double()
    out = 1.5 * F.embedding(tokens, table)
    assert torch.equal(ref.embed(table.detach(), tokens, 1.5), out.detach())
    (g,) = torch.autograd.grad(out, table, d)
    assert torch.allclose(ref.embed_backward(d, tokens, 9, 1.5)[0], g, rtol=1e-12, atol=1e-12)
    # a matrix with orthonormal rows is a fixed point of (1.5, -0.5, 0) up to its scale
    q = torch.linalg.qr(torch.randn(20, 6, generator=gen).double())[0].mT
    out, _ = ref.orthogonalize(q, 12, (1.5, -0.5, 0.0), 0.0)
    assert torch.allclose(out, q, atol=1e-9)
