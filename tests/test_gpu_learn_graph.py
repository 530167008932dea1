"""The learned parts inside a CUDA graph: replays follow their inputs."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_captured_calls_follow_their_inputs():
    from splat_rendering_gb300 import pulsar as pl
    ops = pl.Learner(workspace_bytes=1 << 27)
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    table, grad = r(300, 16), r(9000, 16)
    tokens = torch.randint(-1, 300, (9000,), generator=gen).cuda()
    small, large = r(1, 900, 16), r(2, 40_000, 16)
    w, b = r(16), r(16)
    mats, wide = r(4, 64, 64), r(400, 300)

    def step():
        outs = [ops.embed(table, tokens, 2.0), ops.embed_backward(grad, tokens, 300, 2.0)]
        for x in (small, large):
            y, stats = ops.group_norm(x, 4, w, b, act="silu")
            outs += [y, stats, *ops.group_norm_backward(y, x, stats, 4, w, b, "silu")]
        return outs + [ops.orthogonalize(mats), ops.orthogonalize(wide)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        for t in (table, grad, small, large, w, b, mats, wide):
            t.copy_(r(*t.shape))
        tokens.copy_(torch.randint(-1, 300, (9000,), generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(captured, step()):
            assert torch.equal(got, want)
    ops.status()
    ops.close()


def test_two_handles_on_two_streams():
    """Handles share nothing: the same work on two streams at once."""
    from splat_rendering_gb300 import pulsar as pl
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(1, 60_000, 16, generator=gen).cuda()
    g = torch.randn(300, 500, generator=gen).cuda()
    grad = torch.randn(60_000, 16, generator=gen).cuda()
    tokens = torch.randint(0, 999, (60_000,), generator=gen).cuda()
    handles = [pl.Learner(workspace_bytes=1 << 26) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]

    def work(o):
        y, stats = o.group_norm(x, 2, act="relu")
        return [y, stats, o.orthogonalize(g), o.embed_backward(grad, tokens, 999)]

    want = work(handles[0])
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for o, s in zip(handles, streams):
            with torch.cuda.stream(s):
                got.append(work(o))
    torch.cuda.synchronize()
    for outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    for o in handles:
        o.status()
        o.close()
