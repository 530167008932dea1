"""Norm, linear layers and dropout together, as a network over a feature image uses them: a
pre-norm residual block, forward and backward, in a graph, and on two handles at once."""
from __future__ import annotations

import pytest
import torch

import learn_reference as lref
import linear_reference as ref

pytestmark = pytest.mark.gpu
GROUPS, P_DROP, SEED = 4, 0.2, 99


class Block:
    """y = x + dropout(W2 silu(W1 norm(x) + b1) + b2) of a feature image [images, pixels, C]."""

    def __init__(self, C, hidden, dtype, seed=1, images=1, pixels=900):
        from splat_rendering_gb300 import pulsar as pl
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.x = r(images, pixels, C).to(dtype).cuda()
        self.dy = r(images, pixels, C).to(dtype).cuda()
        self.gamma, self.beta = (1 + 0.2 * r(C)).cuda(), (0.2 * r(C)).cuda()
        self.w1, self.b1 = (r(hidden, C) / C ** 0.5).to(dtype).cuda(), (0.2 * r(hidden)).cuda()
        self.w2, self.b2 = (r(C, hidden) / hidden ** 0.5).to(dtype).cuda(), (0.2 * r(C)).cuda()
        rows = images * pixels
        self.ops = pl.Learner(workspace_bytes=max(
            pl.group_norm_workspace(images, pixels, C, GROUPS),
            pl.linear_workspace(rows, C, hidden, dtype), pl.linear_workspace(rows, hidden, C, dtype)))

    def forward(self, offset=0, counter=None):
        o = self.ops
        h, stats = o.group_norm(self.x, GROUPS, self.gamma, self.beta)
        a, z = o.linear(h, self.w1, self.b1, act="silu", want_pre=True)
        u, _ = o.linear(a, self.w2, self.b2)
        y = o.dropout(u, P_DROP, SEED, offset, counter, residual=self.x)
        return y, (h, stats, a, z)

    def backward(self, saved, offset=0, counter=None):
        o = self.ops
        h, stats, a, z = saved
        du = o.dropout(self.dy, P_DROP, SEED, offset, counter)
        da, dw2, db2 = o.linear_backward(du, a, self.w2)
        dh, dw1, db1 = o.linear_backward(da, h, self.w1, z, act="silu")
        dx, dgamma, dbeta = o.group_norm_backward(dh, self.x, stats, GROUPS, self.gamma, self.beta)
        return dx + self.dy, dgamma, dbeta, dw1, db1, dw2, db2

    def exact(self, offset=0):
        """y and the gradients in 64 bits, by autograd."""
        F = torch.nn.functional
        leaf = lambda t: t.cpu().double().requires_grad_()  # noqa: E731
        x, ga, be, w1, b1, w2, b2 = map(leaf, (self.x, self.gamma, self.beta, self.w1, self.b1,
                                               self.w2, self.b2))
        h = F.group_norm(x.transpose(1, 2), GROUPS, ga, be, 1e-5).transpose(1, 2)
        u = F.linear(F.silu(F.linear(h, w1, b1)), w2, b2)
        keep = (ref.dropout_words(u.numel(), SEED, offset) >= round(P_DROP * 2 ** 32)).view(u.shape)
        y = x + torch.where(keep, u / (1 - P_DROP), 0.0)
        grads = torch.autograd.grad(y, (x, ga, be, w1, b1, w2, b2), self.dy.cpu().double())
        return y.detach(), grads


@pytest.mark.parametrize("C,hidden", [(16, 64), (64, 300), (24, 17)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_block_against_64_bits(C, hidden, dtype):
    """In 32 bits four products deep, each within 1e-6 of its norm, and sums of a thousand rows:
    1e-5.  In 16 bits every intermediate is rounded (rms 2^-9.3 of it), some six of them one after
    another: 3 percent holds ten of their worst."""
    b = Block(C, hidden, dtype)
    y, saved = b.forward(offset=5)
    got = b.backward(saved, offset=5)
    want_y, want = b.exact(offset=5)
    tol = 1e-5 if dtype == torch.float32 else 3e-2
    for name, g, v in zip(("y", "dx", "dgamma", "dbeta", "dw1", "db1", "dw2", "db2"),
                          (y, *got), (want_y, *want)):
        e = float((g.cpu().double() - v).norm() / v.norm())
        assert e <= tol, (name, e)
    b.ops.status()
    b.ops.close()


def test_block_in_a_graph_follows_its_inputs():
    """Forward and backward captured; a counter gives every replay its own numbers."""
    b = Block(16, 64, torch.float32, pixels=2000)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    b.backward(b.forward(3, counter)[1], 3, counter)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, saved = b.forward(3, counter)
        grads = b.backward(saved, 3, counter)
        counter += 8000
    g = torch.Generator().manual_seed(5)
    for k in range(3):
        for t in (b.x, b.dy, b.w1, b.b1, b.w2, b.b2, b.gamma, b.beta):
            t.copy_(torch.randn(t.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want_y, want_saved = b.forward(3 + 8000 * k)
        want = b.backward(want_saved, 3 + 8000 * k)
        for p, q in zip((y, *grads), (want_y, *want)):
            assert torch.equal(p, q)
    b.ops.status()
    b.ops.close()


@pytest.mark.parametrize("shape", [(64, 64), (300, 500)], ids=["narrow", "wide"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_two_handles_on_two_streams(shape, dtype):
    """Handles share nothing: the same work on two streams at once."""
    blocks = [Block(shape[0], shape[1], dtype, seed=7, pixels=30_000) for _ in range(2)]
    y, saved = blocks[0].forward()
    want = (y, *blocks[0].backward(saved))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                y, saved = b.forward()
                got.append((y, *b.backward(saved)))
    torch.cuda.synchronize()
    for outs in got:
        assert all(torch.equal(p, q) for p, q in zip(outs, want))
    for b in blocks:
        b.ops.status()
        b.ops.close()


def test_two_graphs_of_one_handle_replayed_in_turn():
    """They share the workspace, and so are replayed in order on one stream."""
    from splat_rendering_gb300 import pulsar as pl
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    ops = pl.Learner(workspace_bytes=1 << 27)
    x, dy, w = r(3000, 200), r(3000, 130), r(130, 200)
    xn, dn, wn = r(3000, 40), r(3000, 24), r(24, 40)
    calls = [lambda: ops.linear_backward(dy, x, w), lambda: ops.linear_backward(dn, xn, wn)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(c())
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o, v in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(o, v))
    ops.status()
    ops.close()


def test_outputs_survive_the_other_stream():
    """Outputs of a call on a given stream come from its memory."""
    from splat_rendering_gb300 import pulsar as pl
    g = torch.Generator().manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    ops = pl.Learner(workspace_bytes=1 << 27)
    x, w, b, dy = r(20_000, 48), r(70, 48), r(70), r(20_000, 70)

    def calls(**kw):
        y, z = ops.linear(x, w, b, act="silu", want_pre=True, **kw)
        return [y, z, *ops.linear_backward(dy, x, w, z, act="silu", **kw),
                ops.dropout(x, 0.3, 1, **kw)]

    want = calls()
    torch.cuda.synchronize()
    for t in want:
        busy = torch.empty(t.numel(), device="cuda")
        torch.cuda._sleep(20_000_000)
        busy.fill_(7.0)
        del busy
    s = torch.cuda.Stream()
    got = calls(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    ops.status()
    ops.close()


def test_norm_of_a_linear_layer_agrees_with_its_definition():
    """The layers' outputs feed one another without conversions: a norm of a layer's output."""
    b = Block(16, 64, torch.float32)
    _, (h, stats, a, z) = b.forward()
    want, _, bound, _ = lref.group_norm(b.x.cpu(), GROUPS, b.gamma.cpu(), b.beta.cpu(), 1e-5, "none")
    assert not lref.outside(h, want, bound).any()
    (_, z_want), (_, e_z) = ref.linear(h.cpu(), b.w1.cpu(), b.b1.cpu(), None, "silu")
    assert not ref.outside(z, z_want, e_z).any()
    b.ops.close()
