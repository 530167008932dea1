"""Learns a codebook of sphere features, a feature norm and a shading network
through the renderer: every learned part of one training step.

    tokens -> embed -> features [n, 16] -> render -> image [H, W, 16]
           -> group norm + SiLU -> shading MLP -> rgb [H, W, 3] -> loss

and back: shading, norm, renderer and codebook gradients; the network's
matrices take orthogonalised updates, everything else plain gradient steps.
The target is the image of a hidden codebook, so the loss can fall.

    python examples/learn_codebook.py [--steps 60] [--spheres 20000] [--size 256]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from splat_rendering_gb300 import pulsar as pl, scenes  # noqa: E402

CHANNELS, GROUPS = 16, 4
# the shading MLP's matrices in its flat parameters: (offset, rows, columns)
MATRICES = ((0, 64, 19), (64 * 19 + 64, 64, 64), (64 * 19 + 64 + 64 * 64 + 64, 3, 64))


class Model:
    """The learned parts and the handles that run them."""

    def __init__(self, spheres: int, rows: int, size: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        sc = scenes.random_scene(seed, spheres, size, size, channels=CHANNELS, n_track=8,
                                 rrange=(0.02, 0.1))
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.pos, self.radius, self.opacity, self.bg = map(up, (sc.pos, sc.radius, sc.opacity, sc.bg))
        self.cam, self.prm = pl.camera(sc.cameras[0]), pl.params(sc.params)
        self.rows, self.size = rows, size
        self.tokens = torch.randint(0, rows, (spheres,), generator=g).to(torch.int32).cuda()
        self.codebook = torch.randn(rows, CHANNELS, generator=g).cuda()
        self.gamma, self.beta = torch.ones(CHANNELS).cuda(), torch.zeros(CHANNELS).cuda()
        self.mlp = torch.from_numpy(scenes.shading_mlp(seed)).cuda()
        self.renderer = pl.Renderer(spheres, 64 * spheres + 65536, size, size, CHANNELS, 8)
        need = [pl.embed_workspace(spheres, rows, CHANNELS),
                pl.group_norm_workspace(1, size * size, CHANNELS, GROUPS)]
        need += [pl.orthogonalize_workspace(1, m, n, torch.float32) for _, m, n in MATRICES]
        self.ops = pl.Learner(workspace_bytes=max(need))

    def forward(self):
        """rgb [H, W, 3]; keeps what the backward pass reads."""
        features = self.ops.embed(self.codebook, self.tokens)
        image = self.renderer.render(self.pos, self.radius, self.opacity, features, self.cam,
                                     self.prm, self.bg)
        x = image.view(1, self.size, self.size, CHANNELS)
        y, stats = self.ops.group_norm(x, GROUPS, self.gamma, self.beta, act="silu")
        rgb = self.renderer.shade(y[0], self.mlp)
        self._saved = x, y, stats
        return rgb

    def backward(self, grad_rgb):
        """Gradients of the codebook, gamma, beta and the flat MLP parameters."""
        x, y, stats = self._saved
        grad_y, grad_mlp = self.renderer.shade_backward(y[0], self.mlp, grad_rgb)
        grad_x, grad_gamma, grad_beta = self.ops.group_norm_backward(
            grad_y.view_as(x), x, stats, GROUPS, self.gamma, self.beta, act="silu")
        grads = self.renderer.backward(grad_x[0], want=("features",))
        grad_codebook = self.ops.embed_backward(grads["features"], self.tokens, self.rows)
        return grad_codebook, grad_gamma, grad_beta, grad_mlp

    def step(self, grads, rate: float):
        grad_codebook, grad_gamma, grad_beta, grad_mlp = grads
        update = grad_mlp.clone()
        for at, m, n in MATRICES:
            w = slice(at, at + m * n)
            self.ops.orthogonalize(grad_mlp[w].view(m, n), out=update[w].view(m, n))
        self.mlp -= rate * update
        scale = lambda g: g / (g.norm() + 1e-12) * g.numel() ** 0.5  # noqa: E731
        self.codebook -= rate * scale(grad_codebook)
        self.gamma -= 0.1 * rate * scale(grad_gamma)
        self.beta -= 0.1 * rate * scale(grad_beta)

    def close(self):
        self.renderer.close()
        self.ops.close()


def train(steps: int = 60, spheres: int = 20_000, rows: int = 256, size: int = 256,
          rate: float = 0.02, seed: int = 0):
    """Losses of `steps` steps towards the image of a hidden codebook."""
    model = Model(spheres, rows, size, seed)
    hidden = model.codebook.clone()
    target = model.forward()
    g = torch.Generator().manual_seed(seed + 1)
    model.codebook = hidden + torch.randn(rows, CHANNELS, generator=g).cuda()
    model.mlp = model.mlp * (1.0 + 0.1 * torch.randn(model.mlp.shape, generator=g).cuda())
    losses = []
    for _ in range(steps):
        diff = model.forward() - target
        losses.append((diff * diff).mean())
        model.step(model.backward(diff * (2.0 / diff.numel())), rate)
    model.renderer.status()
    model.ops.status()
    model.close()
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--spheres", type=int, default=20_000)
    ap.add_argument("--rows", type=int, default=256)
    ap.add_argument("--size", type=int, default=256)
    a = ap.parse_args()
    out = train(a.steps, a.spheres, a.rows, a.size)
    for i in range(0, len(out), max(1, len(out) // 10)):
        print(f"step {i:4d}  loss {out[i]:.6f}")
    print(f"last      loss {out[-1]:.6f}")
