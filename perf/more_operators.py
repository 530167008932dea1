"""Workloads of the dense-layer operators: a linear layer with its bias,
activation and residual in one call, its gradients, and dropout from a
counter-based generator.

`listed()` and `draw()` give cases, `prepare()` their inputs on the GPU,
`run()` one pass through an operator -- in elementary torch operations in 32
bits, or, with `own` set, through splat_rendering_gb300.pulsar.Learner --
`exact()` the same outputs from the definitions in 64 bits, and `work()` the
bytes and operations a pass cannot do without.

    linear           z = x W^T + b,   y = act(z) + residual
    linear_backward  dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum of dz's rows
    dropout          y_i = [u_i >= p] x_i / (1 - p) + residual_i,
                     u_i = word i mod 4 of Philox4x32-7(seed, offset + i / 4) / 2^32
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one token through a large layer: serving, bound by reading the weights
        _linear("linear_token", "linear", 1, 4096, 2048, "bf16", "silu"),
        # the 40 x 24 feature image of 16 channels into 64 hidden units: latency
        _linear("linear_tiny", "linear", 960, 16, 64, "f32", "silu"),
        # a hidden layer of a per-pixel network over a 1024 x 1024 image
        _linear("linear_frame", "linear", 1024 * 1024, 64, 64, "f32", "silu"),
        # the same in 16 bits over six cameras at a quarter of 1920 x 1080, with a skip connection
        _linear("linear_rig", "linear", 6 * 480 * 270, 64, 64, "bf16", "relu", residual=True),
        # a conditioning text's wide layer: an odd number of tokens, bound by the products
        _linear("linear_text", "linear", 16_381, 1024, 4096, "bf16", "silu"),
        # gradients of an odd, oblong layer in 32 bits
        _linear("linear_back_odd", "linear_backward", 4001, 1500, 509, "f32", "none"),
        # gradients of the three large ones
        _linear("linear_back_frame", "linear_backward", 1024 * 1024, 64, 64, "f32", "silu"),
        _linear("linear_back_rig", "linear_backward", 6 * 480 * 270, 64, 64, "bf16", "relu"),
        _linear("linear_back_text", "linear_backward", 16_381, 1024, 4096, "bf16", "silu"),
        # dropout on the hidden units of the 40 x 24 image: latency
        _dropout("dropout_tiny", 960, 64, "f32", 0.1, False),
        # on a 1024 x 1024 image of 16 channels inside a skip connection
        _dropout("dropout_frame", 1024 * 1024, 16, "f32", 0.1, True),
        # on the rig's hidden units in 16 bits (its gradient is the same call on dy)
        _dropout("dropout_rig", 6 * 480 * 270, 64, "bf16", 0.5, False),
    ]


def _linear(name, op, rows, inputs, outputs, dtype, act, bias=True, residual=False):
    return {"name": name, "op": op, "rows": rows, "inputs": inputs, "outputs": outputs,
            "dtype": dtype, "act": act, "bias": bias, "residual": residual}


def _dropout(name, rows, channels, dtype, p, residual):
    return {"name": name, "op": "dropout", "rows": rows, "channels": channels, "dtype": dtype,
            "p": p, "residual": residual}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "linear_backward", "dropout"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "dropout":
        channels = _log_int(rng, 1, 1024)
        rows = _log_int(rng, 1, 49_000_000 // channels // (2 if dtype == "f32" else 1))
        case = _dropout("", rows, channels, dtype, round(rng.uniform(0.0, 0.9), 3),
                        rng.random() < 0.5)
    else:
        k, n = _log_int(rng, 1, 4096), _log_int(rng, 1, 4096)
        most = min(1024 * 1024, 2 ** 26 // max(k, n), 16_381 * 1024 * 4096 // (k * n))
        act = rng.choice(["none", "silu", "relu"])
        case = _linear("", op, _log_int(rng, 1, most), k, n, dtype, act,
                       bias=op == "linear_backward" or rng.random() < 0.7,
                       residual=op == "linear" and rng.random() < 0.3)
    del case["name"]
    return case


# ----------------------------------------------------------------- inputs --
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    dtype = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = dict(case)
    if case["op"] == "dropout":
        shape = case["rows"], case["channels"]
        s["x"] = normal(*shape).to(dtype)
        s["skip"] = normal(*shape).to(dtype) if case["residual"] else None
        # what a training program counts up: a seed of its own, and the numbers drawn so far
        s["seed"] = int(torch.randint(0, 2 ** 62, (1,), device="cuda", generator=g))
        s["offset"] = int(torch.randint(0, 2 ** 40, (1,), device="cuda", generator=g))
        return s
    M, K, N = case["rows"], case["inputs"], case["outputs"]
    s["x"] = normal(M, K).to(dtype)
    s["weight"] = normal(N, K).mul_(1.0 / math.sqrt(K)).to(dtype)
    s["b"] = 0.2 * normal(N) if case["bias"] else None
    if case["op"] == "linear":
        s["skip"] = normal(M, N).to(dtype) if case["residual"] else None
        return s
    s["grad_y"] = normal(M, N).mul_(1e-2).to(dtype)
    # what the forward pass left behind: z, where the activation's gradient asks for it
    s["z"] = None
    if case["act"] != "none":
        s["z"] = (s["x"].float() @ s["weight"].float().T + s["b"]).to(dtype)
    return s


# ------------------------------------------------------------------- runs --
_learner = None


def _ops(nbytes):
    """The handle a program keeps for its operators: one, grown when a call needs more."""
    global _learner
    from splat_rendering_gb300 import pulsar as pl
    if _learner is None or _learner.workspace_bytes < nbytes:
        _learner = None
        _learner = pl.Learner(workspace_bytes=max(int(nbytes), 1 << 28))
    return _learner


def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    from splat_rendering_gb300 import pulsar as pl
    if s["op"] == "dropout":
        return _ops(0).dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["skip"])
    ops = _ops(pl.linear_workspace(s["rows"], s["inputs"], s["outputs"], s["x"].dtype))
    if s["op"] == "linear":
        return ops.linear(s["x"], s["weight"], s["b"], s["skip"], act=s["act"])[0]
    return ops.linear_backward(s["grad_y"], s["x"], s["weight"], s["z"], act=s["act"])


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _plain_linear(s):
    y = torch.matmul(s["x"].float(), s["weight"].float().T)
    if s["b"] is not None:
        y = y + s["b"]
    if s["act"] == "silu":
        y = y * _sigmoid(y)
    elif s["act"] == "relu":
        y = torch.where(y > 0, y, 0.0)
    if s["skip"] is not None:
        y = y + s["skip"].float()
    return y.to(s["x"].dtype)


def _plain_linear_backward(s):
    dz = s["grad_y"].float()
    if s["act"] == "silu":
        z = s["z"].float()
        q = _sigmoid(z)
        dz = dz * (q * (1.0 + z * (1.0 - q)))
    elif s["act"] == "relu":
        dz = torch.where(s["z"].float() > 0, dz, 0.0)
    dx = torch.matmul(dz, s["weight"].float())
    dw = torch.matmul(dz.T, s["x"].float())
    return dx.to(s["x"].dtype), dw.to(s["x"].dtype), dz.sum(dim=0)


_MASK = 0xFFFFFFFF


def _plain_dropout(s):
    n = s["x"].numel()
    # Philox4x32 with 7 rounds: a counter's words are multiplied, swapped and keyed
    counter = torch.arange((n + 3) // 4, device="cuda") + s["offset"]
    c0, c1 = counter & _MASK, counter >> 32
    c2, c3 = torch.zeros_like(c0), torch.zeros_like(c0)
    k0, k1 = s["seed"] & _MASK, s["seed"] >> 32
    for _ in range(7):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((p1 >> 32) & _MASK) ^ c1 ^ k0, p1 & _MASK,
                          ((p0 >> 32) & _MASK) ^ c3 ^ k1, p0 & _MASK)
        k0, k1 = (k0 + 0x9E3779B9) & _MASK, (k1 + 0xBB67AE85) & _MASK
    words = torch.stack([c0, c1, c2, c3], -1).view(-1)[:n].view(s["x"].shape)
    keep = words >= round(s["p"] * 2 ** 32)
    y = torch.where(keep, s["x"].float() * (1.0 / (1.0 - s["p"])), 0.0)
    if s["skip"] is not None:
        y = y + s["skip"].float()
    return y.to(s["x"].dtype)


_PLAIN = {"linear": _plain_linear, "linear_backward": _plain_linear_backward,
          "dropout": _plain_dropout}


# -------------------------------------------------------------- 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        return _exact_dropout(s)
    F = torch.nn.functional
    act = {"none": lambda v: v * 1.0, "silu": F.silu, "relu": torch.relu}[case["act"]]
    x, w = s["x"].double(), s["weight"].double()
    if case["op"] == "linear":
        y = act(F.linear(x, w, None if s["b"] is None else s["b"].double()))
        return y if s["skip"] is None else y.add_(s["skip"].double())
    dz = s["grad_y"].double()
    if s["z"] is not None:
        z = s["z"].double().requires_grad_()
        (dz,) = torch.autograd.grad(act(z), z, dz)
    return (torch.einsum("mn,nk->mk", dz, w), torch.einsum("mn,mk->nk", dz, x),
            torch.einsum("mn->n", dz))


def _high_low(a, b):
    """The halves of the 64-bit product of a constant and 32-bit words, by 16-bit digits."""
    a1, a0, b1, b0 = a >> 16, a & 0xFFFF, b >> 16, b & 0xFFFF
    low, mid = a0 * b0, a1 * b0 + ((a0 * b0) >> 16)
    mid0 = (mid & 0xFFFF) + a0 * b1
    return a1 * b1 + (mid >> 16) + (mid0 >> 16), ((mid0 & 0xFFFF) << 16) | (low & 0xFFFF)


def _exact_dropout(s):
    x = s["x"].reshape(-1)
    n, blocks = x.numel(), -(-x.numel() // 4)
    at = s["offset"] + torch.arange(blocks, device=x.device)
    ctr = [at % 2 ** 32, at // 2 ** 32, at * 0, at * 0]
    for r in range(7):
        key = [(s["seed"] + r * 0x9E3779B9) % 2 ** 32, (s["seed"] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
        (h0, l0), (h1, l1) = _high_low(0xD2511F53, ctr[0]), _high_low(0xCD9E8D57, ctr[2])
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
    words = torch.empty(blocks, 4, dtype=torch.int64, device=x.device)
    for j in range(4):
        words[:, j] = ctr[j]
    out = x.double() / (1.0 - s["p"])
    out[words.reshape(-1)[:n] < round(s["p"] * 2 ** 32)] = 0.0
    out = out.view(s["x"].shape)
    return out if s["skip"] is None else out.add_(s["skip"].double())


# ------------------------------------------------------------------- work --
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "dropout":
        n = case["rows"] * case["channels"]
        return {"bytes": n * size * (3 if case["residual"] else 2), "flops": 2 * n}
    M, K, N = case["rows"], case["inputs"], case["outputs"]
    product = 2 * M * N * K
    if case["op"] == "linear":
        outs = M * N * (2 if case["residual"] else 1)
        return {"bytes": size * (M * K + N * K + outs) + 4 * N * case["bias"], "flops": product}
    # dy and, for an activation, z; x and dx; W and dW; db
    ins = M * N * (1 if case["act"] == "none" else 2)
    return {"bytes": size * (ins + 2 * M * K + 2 * N * K) + 4 * N, "flops": 2 * product}
