"""Outputs that a call allocates come from the memory of the stream it runs on."""
from __future__ import annotations

import contextlib

import numpy as np
import pytest
import torch


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_allocation_follows_the_stream(monkeypatch):
    """Without a GPU: which stream is current where the tensor is made."""
    from splat_rendering_gb300 import pulsar as pl
    current, made = [_Stream(11)], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: _Stream(h))
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (made.append(current[-1].cuda_stream),
                                                        empty(1))[1])
    ops = object.__new__(pl.Learner)
    ops.handle, ops.device, ops._dev, ops._torch = 0, 0, "cuda:0", torch
    for given, want in ((None, 11), (_Stream(11), 11), (_Stream(5), 5), (7, 7), (0, 0)):
        ops._out(None, "out", (1,), torch.float32, given)
        assert made.pop() == want and not made


def _busy(nbytes):
    """Fills a tensor late on the current stream and frees it: its block may be
    handed out again on this stream, where the next use comes after the fill."""
    t = torch.empty(nbytes // 4, device="cuda")
    torch.cuda._sleep(20_000_000)   # some 10 ms
    t.fill_(7.0)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_learner_outputs_survive_the_other_stream(handle):
    from splat_rendering_gb300 import pulsar as pl
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(1, 30_000, 16, generator=gen).cuda()
    table = torch.randn(100, 16, generator=gen).cuda()
    tokens = torch.randint(0, 100, (30_000,), generator=gen).cuda()
    g = torch.randn(2, 300, 400, generator=gen).cuda()
    ops = pl.Learner(workspace_bytes=1 << 26)
    s = torch.cuda.Stream()
    arg = s.cuda_stream if handle else s
    _, stats = ops.group_norm(x, 4)

    def calls(**kw):
        return [ops.embed(table, tokens, **kw), ops.embed_backward(x[0], tokens, 100, **kw),
                *ops.group_norm(x, 4, **kw), *ops.group_norm_backward(x, x, stats, 4, **kw),
                ops.orthogonalize(g, **kw)]

    want = calls()
    torch.cuda.synchronize()
    sizes = [t.numel() * 4 for t in want]
    for n in sizes:
        _busy(n)
    got = calls(stream=arg)
    s.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    ops.status()
    ops.close()


@pytest.mark.gpu
def test_renderer_outputs_survive_the_other_stream():
    from splat_rendering_gb300 import pulsar as pl, scenes
    sc = scenes.tiny()
    cam, p = sc.cameras[0], sc.params
    r = pl.Renderer(max_spheres=sc.n, max_pairs=64 * sc.n, max_width=cam.width,
                    max_height=cam.height, max_channels=p.channels, max_track=p.n_track)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    args = (t(sc.pos), t(sc.radius), t(sc.opacity), t(sc.features), pl.camera(cam), pl.params(p),
            t(sc.bg))
    grad = t(sc.grad_images[0])

    def calls(**kw):
        image = r.render(*args, **kw)
        return [image, *r.backward(grad, **kw).values()]

    want = calls()
    torch.cuda.synchronize()
    for v in want:
        _busy(v.numel() * 4)
    s = torch.cuda.Stream()
    got = calls(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
    for a, b in zip(got[1:], want[1:]):   # (their sums' order varies)
        assert (a - b).abs().max() <= 1e-3 * b.abs().max()
    r.status()
    r.close()
