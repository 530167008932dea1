"""Tensors of more than 2^31 elements: every offset of the learned parts is 64
bits wide.  The inputs repeat, so that the results are known everywhere."""
from __future__ import annotations

import pytest
import torch

import learn_reference as ref

pytestmark = pytest.mark.gpu


def _free(nbytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < nbytes:
        pytest.skip("not enough device memory")


def test_embedding():
    from splat_rendering_gb300 import pulsar as pl
    n, rows, dim = 2_100_000, 7, 1032
    assert n * dim > 1 << 31
    _free(16 << 30)
    gen = torch.Generator().manual_seed(1)
    table = torch.randint(-2, 3, (rows, dim), generator=gen).to(torch.bfloat16).cuda()
    tokens = (torch.arange(n, device="cuda") * 5) % (rows + 1) - 1   # every eighth masked
    ops = pl.Learner(workspace_bytes=pl.embed_workspace(n, rows, dim))
    out = ops.embed(table, tokens, 2.0)
    for at in (0, n // 2, n - 1000):
        t = tokens[at:at + 1000]
        want = torch.where((t >= 0)[:, None], 2.0 * table[t.clamp(min=0)], 0.0)
        assert torch.equal(out[at:at + 1000], want)
    # the sums of small whole numbers are exact in 32 bits
    grad = ops.embed_backward(out, tokens, rows, 0.5)
    count = torch.bincount(tokens[tokens >= 0], minlength=rows).float()
    assert torch.equal(grad, (count[:, None] * table.float()).to(torch.bfloat16))
    assert ops.status() == 0
    ops.close()


def test_group_norm():
    from splat_rendering_gb300 import pulsar as pl
    C, G, reps, period = 16, 4, 135_000, 1000
    assert reps * period * C > 1 << 31
    _free(40 << 30)
    gen = torch.Generator().manual_seed(2)
    x1, dy1 = (torch.randn(1, period, C, generator=gen).to(torch.bfloat16) for _ in range(2))
    w, b = 1 + 0.3 * torch.randn(C, generator=gen), 0.3 * torch.randn(C, generator=gen)
    x = x1.cuda().repeat(1, reps, 1)
    dy = dy1.cuda().repeat(1, reps, 1)
    ops = pl.Learner(workspace_bytes=pl.group_norm_workspace(1, reps * period, C, G))
    y, stats = ops.group_norm(x, G, w.cuda(), b.cuda(), act="silu")
    want, s_want, e_y, e_s = ref.group_norm(x1, G, w, b, 1e-5, "silu")
    # (a thread's sums are of 64 pixels at a time, whatever the image; the
    # joins are some tens of levels deeper than at the small sizes)
    assert not ref.outside(stats, s_want, 4 * e_s).any()
    assert not ref.outside(y[:, :period], want, 4 * e_y).any()
    pieces = y.view(reps, period, C)
    assert all(torch.equal(pieces[i], pieces[0]) for i in (1, reps // 2, reps - 1))
    assert torch.equal(pieces[1:].amax(0), pieces[0]) and torch.equal(pieces[1:].amin(0), pieces[0])
    dx, dw, db = ops.group_norm_backward(dy, x, stats, G, w.cuda(), b.cuda(), "silu")
    (dx1, dw1, db1), (e_dx, e_dw, e_db) = ref.group_norm_backward(dy1, x1, stats.cpu(), G, w, b, "silu")
    assert not ref.outside(dx[:, :period], dx1, 4 * e_dx).any()
    assert not ref.outside(dw / reps, dw1, 4 * e_dw).any()
    assert not ref.outside(db / reps, db1, 4 * e_db).any()
    pieces = dx.view(reps, period, C)
    assert torch.equal(pieces[1:].amax(0), pieces[0]) and torch.equal(pieces[1:].amin(0), pieces[0])
    assert ops.status() == 0
    ops.close()


def test_orthogonalize_batch():
    from splat_rendering_gb300 import pulsar as pl
    B, m, n = 40_000, 60, 900
    assert B * m * n > 1 << 31
    _free(40 << 30)
    one = torch.randn(m, n, generator=torch.Generator().manual_seed(3)).cuda()
    ops = pl.Learner(workspace_bytes=pl.orthogonalize_workspace(B, m, n, one.dtype))
    grad = one.repeat(B, 1, 1)
    out = ops.orthogonalize(grad, out=grad)
    alone = ops.orthogonalize(one[None].repeat(200, 1, 1))   # the same form: many matrices
    assert torch.equal(out[0], alone[0])
    assert all(torch.equal(out[i], out[0]) for i in (1, B // 2, B - 1))
    assert torch.equal(out.amax(0), out[0]) and torch.equal(out.amin(0), out[0])
    assert ops.status() == 0
    ops.close()
