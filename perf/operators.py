"""Workloads of the learned-feature operators: the codebook embedding, the
channels-last group normalisation with its activation, and the Newton-Schulz
orthogonalisation of an update.

`listed()` and `draw()` give cases, `prepare()` their inputs on the GPU,
`run()` one pass through an operator -- in elementary torch operations in 32
bits, or, with `own` set, through splat_rendering_gb300.pulsar.Learner --
`exact()` the same outputs from the definitions in 64 bits, and `work()` the
bytes and operations a pass cannot do without.

    embed           out_i = s table[t_i]                          (t_i < 0: a zero row)
    embed_backward  dtable_v = s sum_{i: t_i = v} dout_i
    norm            z = gamma_c (x - mu_g) / sqrt(var_g + eps) + beta_c,  y = act(z)
    norm_backward   dx, dgamma, dbeta of sum <dy, y>
    orth            X_0 = G / (|G|_F + eps),  X' = a X + (b A + c A^2) X,  A = X X^T
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5          # of the group norm
ORTH_EPS = 1e-7     # of the orthogonalisation
ORTH_COEFFS = (3.4445, -4.775, 2.0315)
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the spheres of a small scene read their colour from a 256-entry codebook: latency
        _embed("embed_tiny", "embed", 1000, 256, 3, "f32", "i32"),
        # a million spheres with 16-channel features from a codebook of 8192, and its gradient
        _embed("embed_spheres", "embed", 1_000_000, 8192, 16, "f32", "i32"),
        _embed("embed_back_spheres", "embed_backward", 1_000_000, 8192, 16, "f32", "i32"),
        # wide rows, a large table, an odd number of tokens, 64-bit tokens: a conditioning text
        _embed("embed_back_wide", "embed_backward", 16_381, 50_000, 1024, "bf16", "i64"),
        # a 40 x 24 feature image, the smallest frame: latency
        _norm("norm_tiny", "norm", 1, 24 * 40, 16, 4, "f32", "silu"),
        # the 1024 x 1024 feature image of 16 channels, both directions
        _norm("norm_frame", "norm", 1, 1024 * 1024, 16, 4, "f32", "silu"),
        _norm("norm_back_frame", "norm_backward", 1, 1024 * 1024, 16, 4, "f32", "silu"),
        # six cameras at a quarter of 1920 x 1080 with 64 channels in 16 bits, both directions
        _norm("norm_rig", "norm", 6, 480 * 270, 64, 8, "bf16", "silu"),
        _norm("norm_back_rig", "norm_backward", 6, 480 * 270, 64, 8, "bf16", "relu"),
        # the updates of eight 64 x 64 layers: latency
        _orth("orth_layers", 8, 64, 64, "f32"),
        # an odd, oblong update in 32 bits
        _orth("orth_oblong", 1, 1500, 509, "f32"),
        # a large layer's update in 16 bits
        _orth("orth_large", 1, 2048, 4096, "bf16"),
    ]


def _embed(name, op, n, rows, dim, dtype, index):
    return {"name": name, "op": op, "n": n, "rows": rows, "dim": dim, "dtype": dtype,
            "index": index}


def _norm(name, op, images, pixels, channels, groups, dtype, act):
    return {"name": name, "op": op, "images": images, "pixels": pixels, "channels": channels,
            "groups": groups, "dtype": dtype, "act": act}


def _orth(name, batch, m, n, dtype):
    return {"name": name, "op": "orth", "batch": batch, "m": m, "n": n, "dtype": dtype}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_backward", "norm", "norm_backward", "orth"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("embed", "embed_backward"):
        dim = _log_int(rng, 1, 1024)
        n = _log_int(rng, 1, min(1_000_000, 16_700_000 // dim))
        rows = _log_int(rng, 1, min(200_000, 51_200_000 // dim))
        case = _embed("", op, n, rows, dim, dtype, rng.choice(["i32", "i64"]))
    elif op in ("norm", "norm_backward"):
        groups = rng.choice([1, 2, 3, 4, 8, 16, 32])
        channels = groups * _log_int(rng, 1, 24)
        images = rng.randint(1, 8)
        # below some 16 values a group, its gradient is what rounding leaves of a cancellation
        pixels = _log_int(rng, 16, min(1024 * 1024, 24_000_000 // (images * channels)))
        case = _norm("", op, images, pixels, channels, groups, dtype,
                     rng.choice(["none", "silu", "relu"]))
    else:
        m, n = _log_int(rng, 1, 2048), _log_int(rng, 1, 4096)
        cost = min(m, n) ** 2 * max(m, n)
        batch = _log_int(rng, 1, max(1, min(16, 2048 * 2048 * 2048 // cost)))
        case = _orth("", batch, m, n, dtype)
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
    if case["op"] in ("embed", "embed_backward"):
        n, rows, dim = case["n"], case["rows"], case["dim"]
        # few entries are popular and most are rare; a token in fifty has no entry (-1)
        u = torch.rand(n, device="cuda", generator=g, dtype=torch.float64)
        t = (u.pow(3) * rows).long().clamp_(max=rows - 1)
        t = torch.randperm(rows, device="cuda", generator=g)[t]
        t[torch.rand(n, device="cuda", generator=g) < 0.02] = -1
        s["tokens"] = t.to(torch.int32 if case["index"] == "i32" else torch.int64)
        s["scale"] = math.sqrt(dim)
        if case["op"] == "embed":
            s["table"] = normal(rows, dim).to(dtype)
        else:
            s["grad_out"] = normal(n, dim).to(dtype)
    elif case["op"] in ("norm", "norm_backward"):
        N, P, C, G = case["images"], case["pixels"], case["channels"], case["groups"]
        x = normal(N, P, C).mul_(0.5 + torch.rand(C, device="cuda", generator=g)).add_(normal(C))
        s["x"] = x.to(dtype)
        s["weight"] = 1.0 + 0.2 * normal(C)
        s["bias"] = 0.2 * normal(C)
        if case["op"] == "norm_backward":
            s["grad_y"] = normal(N, P, C).to(dtype)
            # what the forward pass left behind
            v = s["x"].view(N, P, G, C // G).double()
            var, mean = torch.var_mean(v, dim=(1, 3), correction=0)
            s["stats"] = torch.stack([mean, (var + EPS).rsqrt()], -1).float()
    else:
        B, m, n = case["batch"], case["m"], case["n"]
        # a gradient: some strong directions above a noise floor
        k = max(1, min(m, n) // 8)
        low = torch.matmul(normal(B, m, k), normal(B, k, n))
        s["grad"] = (1e-3 * (low / math.sqrt(k) + 0.5 * normal(B, m, n))).to(dtype)
    return s


# ------------------------------------------------------------------- runs --
_learner = None


def _ops(nbytes):
    """The handle a program keeps for its operators: one, grown when a call needs more."""
    global _learner
    from splat_rendering_gb300 import pulsar as pl
    if _learner is None or _learner.workspace_bytes < nbytes:
        _learner = pl.Learner(workspace_bytes=max(int(nbytes), 1 << 28))
    return _learner


def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    from splat_rendering_gb300 import pulsar as pl
    op = s["op"]
    if op == "embed":
        return _ops(0).embed(s["table"], s["tokens"], s["scale"])
    if op == "embed_backward":
        ops = _ops(pl.embed_workspace(s["n"], s["rows"], s["dim"]))
        return ops.embed_backward(s["grad_out"], s["tokens"], s["rows"], s["scale"])
    if op in ("norm", "norm_backward"):
        ops = _ops(pl.group_norm_workspace(s["images"], s["pixels"], s["channels"], s["groups"]))
        if op == "norm":
            return ops.group_norm(s["x"], s["groups"], s["weight"], s["bias"], EPS, s["act"])
        return ops.group_norm_backward(s["grad_y"], s["x"], s["stats"], s["groups"], s["weight"],
                                       s["bias"], s["act"])
    ops = _ops(pl.orthogonalize_workspace(s["batch"], s["m"], s["n"], s["grad"].dtype))
    return ops.orthogonalize(s["grad"], steps=5, coeffs=ORTH_COEFFS, eps=ORTH_EPS)


def _plain_embed(s):
    t = s["tokens"].long()
    out = s["table"].float()[t.clamp(min=0)] * s["scale"]
    return torch.where((t >= 0)[:, None], out, 0.0).to(s["table"].dtype)


def _plain_embed_backward(s):
    t = s["tokens"].long()
    keep = (t >= 0)[:, None]
    rows = torch.where(keep, s["grad_out"].float(), 0.0)
    out = torch.zeros(s["rows"], s["dim"], device=rows.device)
    out.index_add_(0, t.clamp(min=0), rows)
    return (out * s["scale"]).to(s["grad_out"].dtype)


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _plain_norm(s):
    N, P, C, G = s["images"], s["pixels"], s["channels"], s["groups"]
    x = s["x"].float().view(N, P, G, C // G)
    mean = x.mean(dim=(1, 3), keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(dim=(1, 3), keepdim=True) + EPS)
    z = (d * rstd).view(N, P, C) * s["weight"] + s["bias"]
    if s["act"] == "silu":
        z = z * _sigmoid(z)
    elif s["act"] == "relu":
        z = torch.where(z > 0, z, 0.0)
    return z.to(s["x"].dtype), torch.stack([mean.view(N, G), rstd.view(N, G)], -1)


def _plain_norm_backward(s):
    N, P, C, G = s["images"], s["pixels"], s["channels"], s["groups"]
    mean, rstd = (s["stats"][..., i].view(N, 1, G, 1) for i in (0, 1))
    xhat = ((s["x"].float().view(N, P, G, C // G) - mean) * rstd).view(N, P, C)
    z = xhat * s["weight"] + s["bias"]
    dz = s["grad_y"].float()
    if s["act"] == "silu":
        q = _sigmoid(z)
        dz = dz * (q * (1.0 + z * (1.0 - q)))
    elif s["act"] == "relu":
        dz = torch.where(z > 0, dz, 0.0)
    dbeta = dz.sum(dim=(0, 1))
    dgamma = (dz * xhat).sum(dim=(0, 1))
    dh = (dz * s["weight"]).view(N, P, G, C // G)
    xh = xhat.view(N, P, G, C // G)
    m1 = dh.mean(dim=(1, 3), keepdim=True)
    m2 = (dh * xh).mean(dim=(1, 3), keepdim=True)
    dx = (rstd * (dh - m1 - xh * m2)).view(N, P, C)
    return dx.to(s["x"].dtype), dgamma, dbeta


def _plain_orth(s):
    a, b, c = ORTH_COEFFS
    x = s["grad"].float()
    tall = s["m"] > s["n"]
    if tall:
        x = x.transpose(1, 2)
    x = x / ((x * x).sum(dim=(1, 2), keepdim=True).sqrt() + ORTH_EPS)
    for _ in range(5):
        A = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * A + c * torch.matmul(A, A), x)
    if tall:
        x = x.transpose(1, 2)
    return x.to(s["grad"].dtype).contiguous()


_PLAIN = {"embed": _plain_embed, "embed_backward": _plain_embed_backward, "norm": _plain_norm,
          "norm_backward": _plain_norm_backward, "orth": _plain_orth}


# -------------------------------------------------------------- 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        t = s["tokens"].long()
        padded = torch.cat([s["table"].double(), torch.zeros(1, s["dim"], device="cuda",
                                                            dtype=torch.float64)])
        return s["scale"] * padded[torch.where(t < 0, s["rows"], t)]
    if op == "embed_backward":
        # sorted by token, a row's sum is a difference of the running sums
        t, order = torch.sort(s["tokens"].long(), stable=True)
        run_sum = torch.cumsum(s["grad_out"].double()[order], 0)
        run_sum = torch.cat([torch.zeros_like(run_sum[:1]), run_sum])
        v = torch.arange(s["rows"], device="cuda")
        ends, starts = torch.searchsorted(t, v, right=True), torch.searchsorted(t, v)
        return s["scale"] * (run_sum[ends] - run_sum[starts])
    if op in ("norm", "norm_backward"):
        return _exact_norm(s)
    r, c = min(s["m"], s["n"]), max(s["m"], s["n"])
    if r > 2048 or s["batch"] * r * r * c > 2e10:
        return None
    # X_k = V q_k(L) V^T X_0 with X_0 X_0^T = V L V^T, each factor of q_k at L q_{k-1}^2
    x = s["grad"].double()
    if s["m"] > s["n"]:
        x = x.mT
    x = x / (torch.linalg.matrix_norm(x)[:, None, None] + ORTH_EPS)
    lam, V = torch.linalg.eigh(x @ x.mT)
    q = torch.ones_like(lam)
    for _ in range(5):
        l2 = lam * q * q
        q = q * (ORTH_COEFFS[0] + l2 * (ORTH_COEFFS[1] + ORTH_COEFFS[2] * l2))
    out = (V * q[:, None, :]) @ (V.mT @ x)
    return (out.mT if s["m"] > s["n"] else out).contiguous()


def _exact_norm(s):
    """The definition with each group's elements in a row, image by image."""
    N, P, C, G = s["images"], s["pixels"], s["channels"], s["groups"]
    w, b = s["weight"].double(), s["bias"].double()
    ys, stats, dw, db = [], [], 0.0, 0.0
    for i in range(N):
        x = s["x"][i].double().view(P, G, C // G).transpose(0, 1).reshape(G, -1)
        if s["op"] == "norm":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + EPS) ** -0.5
        else:
            mean, rstd = s["stats"][i].double().unbind(-1)
        h = (x - mean[:, None]) * rstd[:, None]
        hc = h.view(G, P, C // G).transpose(0, 1).reshape(P, C)
        z = (w * hc + b).requires_grad_(s["op"] == "norm_backward")
        y = {"silu": torch.nn.functional.silu, "relu": torch.relu, "none": lambda v: v * 1.0}[
            s["act"]](z)
        if s["op"] == "norm":
            ys.append(y)
            stats.append(torch.stack([mean, rstd], -1))
            continue
        (dz,) = torch.autograd.grad(y, z, s["grad_y"][i].double())
        dw, db = dw + (dz * hc).sum(0), db + dz.sum(0)
        dh = (dz * w).view(P, G, C // G).transpose(0, 1).reshape(G, -1)
        dx = rstd[:, None] * (dh - dh.mean(1, keepdim=True) - h * (dh * h).mean(1, keepdim=True))
        ys.append(dx.view(G, P, C // G).transpose(0, 1).reshape(P, C))
    out = torch.stack(ys)
    return (out, torch.stack(stats)) if s["op"] == "norm" else (out, dw, db)


# ------------------------------------------------------------------- work --
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("embed", "embed_backward"):
        n, rows, dim = case["n"], case["rows"], case["dim"]
        tokens = n * (4 if case["index"] == "i32" else 8)
        # the forward reads each table row that a token names once
        table = (min(n, rows) if case["op"] == "embed" else rows) * dim * size
        return {"bytes": tokens + n * dim * size + table, "flops": n * dim}
    if case["op"] in ("norm", "norm_backward"):
        n = case["images"] * case["pixels"] * case["channels"]
        back = case["op"] == "norm_backward"
        small = 8 * case["images"] * case["groups"] + (16 if back else 8) * case["channels"]
        return {"bytes": n * size * (3 if back else 2) + small, "flops": n * (20 if back else 10)}
    # a step: X X^T and A A^T are symmetric (half of each), and their sum times X is whole
    r, c = min(case["m"], case["n"]), max(case["m"], case["n"])
    return {"bytes": 2 * case["batch"] * r * c * size,
            "flops": 5 * case["batch"] * (r * r * c + r * r * r + 2 * r * r * c)}
