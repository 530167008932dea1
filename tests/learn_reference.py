"""The learned parts' definitions in 64 bits (torch on the CPU), with the
error bounds the GPU tests use; tests only.

U32 is the unit roundoff of float32.  The bounds are worst-case first-order
rounding bounds of the 32-bit arithmetic the kernels do; each function says of
what.  A bfloat16 result is one more rounding, which is monotone: it has to
lie between the roundings of the two ends of the 32-bit bound (`outside`).
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
THREAD_PIXELS = 64   # pixels one thread sums at most at the tested sizes


def outside(got, want, bound):
    """Which entries of `got` (rounded to its type at the end) are none of the
    values within `bound` of `want`."""
    got = got.cpu()
    lo, hi = want - 1.01 * bound - 1e-30, want + 1.01 * bound + 1e-30
    if got.dtype == torch.bfloat16:
        lo, hi = lo.to(got.dtype).double(), hi.to(got.dtype).double()
    return ~((got.double() >= lo) & (got.double() <= hi))


# -------------------------------------------------------------- embedding --
def embed(table, tokens, scale):
    t = tokens.long()
    out = table.double()[t.clamp(min=0, max=table.shape[0] - 1)] * scale
    return torch.where(((t >= 0) & (t < table.shape[0]))[..., None], out, 0.0)


def embed_backward(grad_out, tokens, rows, scale):
    """(gradient, bound): a row of m terms is off by at most (m + 1) U32 of the
    sum of their magnitudes, and by the scaling's rounding."""
    t = tokens.long().reshape(-1)
    keep = (t >= 0) & (t < rows)
    g = grad_out.double().reshape(-1, grad_out.shape[-1])[keep]
    t = t[keep]
    out = torch.zeros(rows, g.shape[1], dtype=torch.float64).index_add_(0, t, g) * scale
    mag = torch.zeros_like(out).index_add_(0, t, g.abs()) * abs(scale)
    m = torch.bincount(t, minlength=rows).double()[:, None]
    return out, (m + 1) * U32 * mag + U32 * out.abs()


# ------------------------------------------------------------- group norm --
def _grouped(v, groups):
    N, C = v.shape[0], v.shape[-1]
    return v.double().reshape(N, -1, groups, C // groups)


def act(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    return torch.relu(z) if name == "relu" else z


def act_grad(z, name):
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return (z > 0).double() if name == "relu" else torch.ones_like(z)


def _params(x, weight, bias):
    C = x.shape[-1]
    w = torch.ones(C, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(C, dtype=torch.float64) if bias is None else bias.double()
    return w, b


def group_norm(x, groups, weight, bias, eps, name):
    """(y, stats, y's bound, stats' bound).  With D = THREAD_PIXELS + 40 the
    depth of the sums and a = max |x - mean| of the group: the mean is off by
    D U32 (|mean| + 2 a); a thread's second moment about its own first value
    by 3 THREAD_PIXELS U32 of it, in all var by
    3 THREAD_PIXELS U32 (2 var + 2 a^2); z by what these two and its own five
    operations do; the activation's slope is at most 1.1, and its own
    exponential and division are good to 8 U32 + 2 U32 |z|."""
    v = _grouped(x, groups)
    mean = v.mean((1, 3), keepdim=True)
    var = ((v - mean) ** 2).mean((1, 3), keepdim=True)
    rstd = (var + eps) ** -0.5
    a = (v - mean).abs().amax((1, 3), keepdim=True)
    h = (v - mean) * rstd
    w, b = _params(x, weight, bias)
    wg, bg = w.reshape(1, 1, groups, -1), b.reshape(1, 1, groups, -1)
    z = wg * h + bg
    D = THREAD_PIXELS + 40
    e_mean = D * U32 * (mean.abs() + 2 * a)
    e_rstd = 3 * THREAD_PIXELS * U32 * (2 * var + 2 * a * a) / (2 * (var + eps)) + 8 * U32
    e_z = wg.abs() * (rstd * e_mean + h.abs() * (e_rstd + 4 * U32)) + 2 * U32 * (z.abs() + bg.abs())
    y = act(z, name)
    e_y = 1.1 * e_z + y.abs() * (9 + 2 * z.abs()) * U32
    stats = torch.stack([mean.flatten(1), rstd.flatten(1)], -1)
    e_stats = torch.stack([e_mean.flatten(1), (rstd * e_rstd).flatten(1)], -1)
    return y.reshape(x.shape), stats, e_y.reshape(x.shape), e_stats


def group_norm_backward(grad_y, x, stats, groups, weight, bias, name):
    """((dx, dw, db), (their bounds)) for the given (mean, rstd).  h and z are
    off by a few U32 of their terms, dz by that times its slope in z (at most
    1 for silu) and its own operations; a sum of terms by D U32 of the sum of
    their magnitudes, D = THREAD_PIXELS + 300 its depth.  A relu whose z is
    within its error of 0 may go either way: there the whole dy is allowed."""
    v, dy = _grouped(x, groups), _grouped(grad_y, groups)
    N, C = x.shape[0], x.shape[-1]
    mean, rstd = (stats.double()[..., i].reshape(N, 1, groups, 1) for i in (0, 1))
    w, b = _params(x, weight, bias)
    wg, bg = w.reshape(1, 1, groups, -1), b.reshape(1, 1, groups, -1)
    h = (v - mean) * rstd
    z = wg * h + bg
    dz = dy * act_grad(z, name)
    e_h = 3 * U32 * h.abs()
    e_z = wg.abs() * e_h + 2 * U32 * (z.abs() + bg.abs())
    slope = {"silu": 1.0, "relu": 0.0, "none": 0.0}[name]
    e_dz = dy.abs() * (slope * e_z + (16 + 4 * z.abs()) * U32 * (name == "silu")) + 2 * U32 * dz.abs()
    if name == "relu":
        e_dz = torch.where(z.abs() <= e_z, dy.abs(), e_dz)
    D = THREAD_PIXELS + 300

    def channels(t):
        return t.sum(1).reshape(N, C).sum(0)

    db, e_db = channels(dz), channels(e_dz) + D * U32 * channels(dz.abs())
    dw = channels(dz * h)
    e_dw = channels(e_dz * h.abs() + dz.abs() * e_h) + D * U32 * channels((dz * h).abs())
    dh, e_dh = wg * dz, wg.abs() * e_dz
    mean_of = lambda t: t.mean((1, 3), keepdim=True)  # noqa: E731
    m1, m2 = mean_of(dh), mean_of(dh * h)
    e_m1 = mean_of(e_dh) + D * U32 * mean_of(dh.abs())
    e_m2 = mean_of(e_dh * h.abs() + dh.abs() * e_h) + D * U32 * mean_of((dh * h).abs())
    dx = rstd * (dh - m1 - h * m2)
    e_dx = rstd * (e_dh + e_m1 + h.abs() * e_m2 + e_h * m2.abs() +
                   4 * U32 * (dh.abs() + m1.abs() + (h * m2).abs()))
    return ((dx.reshape(x.shape), dw, db), (e_dx.reshape(x.shape), e_dw, e_db))


# ------------------------------------------------------ orthogonalisation --
def orthogonalize(grad, steps, coeffs, eps):
    """(result, bound on the 2-norm of each matrix's error).  A product's
    relative error is taken as eta = 2^-20 in 32 bits and 2^-10 in 16 bits
    (operands rounded to 11 bits, a longer sum); a step of it moves
    a X + (b A + c A^2) X by at most (|a| + 3 |b| s^2 + 5 |c| s^4) eta |X|_F
    for the largest singular value s, and later steps amplify that by at most
    the same polynomial's bound on its slope."""
    a, b, c = coeffs
    x = grad.double().reshape(-1, *grad.shape[-2:])
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.mT
    norm = x.pow(2).sum((1, 2), keepdim=True).sqrt()
    x = x / (norm + eps)
    eta = 2.0 ** -10 if grad.dtype == torch.bfloat16 else 2.0 ** -20
    err = eta * x.pow(2).sum((1, 2)).sqrt()
    for _ in range(steps):
        s2 = torch.linalg.matrix_norm(x, 2) ** 2
        slope = abs(a) + 3 * abs(b) * s2 + 5 * abs(c) * s2 * s2
        # the slope's own bound keeps the terms' signs: of p'(s) on [0, s_max]
        g = torch.linspace(0, 1, 257, dtype=torch.float64)[:, None] * s2.sqrt()
        lip = (a + 3 * b * g ** 2 + 5 * c * g ** 4).abs().amax(0)
        lip = torch.maximum(lip, (a + b * g ** 2 + c * g ** 4).abs().amax(0))
        err = lip * err + slope * eta * x.pow(2).sum((1, 2)).sqrt()
        A = x @ x.mT
        x = a * x + (b * A + c * (A @ A)) @ x
    # the root mean square of a rounding to bfloat16 is below 2^-9
    err = err + (2.0 ** -9 if grad.dtype == torch.bfloat16 else 0.0) * x.pow(2).sum((1, 2)).sqrt()
    if tall:
        x = x.mT
    return x.reshape(grad.shape), err.reshape(grad.shape[:-2])
