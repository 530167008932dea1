"""Definitions of the linear layer and of dropout in 64 bits (torch on the CPU
or the GPU), with the error bounds the GPU tests use; tests only.

U32 and UB are half a step of float32 and bfloat16, relative to a value.  A
product of the tensor cores over K adds 16 terms an instruction, each
instruction's sum truncated to 24 bits: off by at most 2 U32 of the sum of the
terms' magnitudes.  In 32 bits eight instructions follow one another before
the sum is drained (16 U32), drained sums are added in float32 (K / 128 and up
to 160 parts of the contraction), and the left-out products of the operands'
parts are at most 2 U32: (16 + K / 128 + 160 + 4) U32.  In 16 bits nothing is
drained: (K / 8 + 160 + 4) U32.  A bfloat16 result is one more rounding, which
is monotone: it lies between the roundings of the bound's two ends.
"""
from __future__ import annotations

import torch

from learn_reference import U32, act, act_grad, outside  # noqa: F401

UB = 2.0 ** -8


def _product_error(dtype, K):
    return (K / 8 + 164 if dtype == torch.bfloat16 else 180 + K / 128) * U32


def linear(x, weight, bias, residual, name):
    """((y, z), (their bounds)).  The activations' slopes are at most 1.1; the exponential and
    the division are good to 8 U32 + 2 U32 |z|."""
    a, w = x.double(), weight.double()
    z, size = a @ w.T, a.abs() @ w.abs().T
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    e_z = _product_error(x.dtype, x.shape[-1]) * size
    y = act(z, name)
    e_y = 1.1 * e_z + (y.abs() * (9 + 2 * z.abs()) * U32 if name == "silu" else 0.0)
    if residual is not None:
        y = y + residual.double()
        e_y = e_y + 2 * U32 * (y.abs() + residual.double().abs())
    return (y, z), (e_y, e_z)


def linear_backward(grad_y, x, weight, pre, name):
    """((dx, dw, db), (their bounds)) for the given z.  dz is off by a few U32 of its terms, and
    in 16 bits by UB as an operand (exact without an activation); db's sums are at most 400 deep
    (rows of a thread, of a block, and of the blocks)."""
    dy, a, w = grad_y.double(), x.double(), weight.double()
    dz = dy
    e_dz = torch.zeros_like(dy)
    if name != "none":
        z = pre.double()
        dz = dy * act_grad(z, name)
        if name == "silu":
            e_dz = dy.abs() * (16 + 4 * z.abs()) * U32 + 2 * U32 * dz.abs()
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    dz, e_dz, a = flat(dz), flat(e_dz), flat(a)
    db = dz.sum(0)
    e_db = e_dz.sum(0) + 400 * U32 * dz.abs().sum(0)
    e_op = e_dz + (UB * dz.abs() if x.dtype == torch.bfloat16 and name != "none" else 0.0)
    mag = dz.abs() + e_op
    dx, dw = dz @ w, dz.T @ a
    e_dx = e_op @ w.abs() + _product_error(x.dtype, w.shape[0]) * (mag @ w.abs())
    e_dw = e_op.T @ a.abs() + _product_error(x.dtype, a.shape[0]) * (mag.T @ a.abs())
    return (dx.reshape(x.shape), dw, db), (e_dx.reshape(x.shape), e_dw, e_db)


_MASK = 0xFFFFFFFF


def philox(counter, key, rounds: int):
    """Words of Philox4x32 for counters [..., 4] and a key (k0, k1), as int64 tensors."""
    c = [v.clone() for v in counter.unbind(-1)]
    k0, k1 = key
    for _ in range(rounds):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57   # (the bits of an unsigned product)
        c = [((p1 >> 32) & _MASK) ^ c[1] ^ k0, p1 & _MASK,
             ((p0 >> 32) & _MASK) ^ c[3] ^ k1, p0 & _MASK]
        k0, k1 = (k0 + 0x9E3779B9) & _MASK, (k1 + 0xBB67AE85) & _MASK
    return torch.stack(c, -1)


def dropout_words(n, seed, offset):
    """The n random words, in order."""
    at = [(offset + b) & ((1 << 64) - 1) for b in range((n + 3) // 4)]
    ctr = torch.tensor([[v & _MASK, v >> 32, 0, 0] for v in at], dtype=torch.int64).reshape(-1, 4)
    return philox(ctr, (seed & _MASK, seed >> 32), 7).reshape(-1)[:n]


def dropout(x, p, seed, offset, residual):
    """(y, keep, bound): the scale, the product and the sum are each rounded."""
    keep = (dropout_words(x.numel(), seed, offset) >= round(p * 2 ** 32)).view(x.shape)
    y = torch.where(keep, x.double() / (1 - p), 0.0)
    e = 2 * U32 * y.abs()
    if residual is not None:
        y = y + residual.double()
        e = e + U32 * y.abs()
    return y, keep, 1.01 * e
