"""The 8-bit path's definitions in 64 bits, on the CPU, for the GPU tests.

16-bit arrays are held as torch CPU tensors (numpy has no bfloat16)."""

import numpy as np
import torch

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.to(torch.float64).numpy()


def nearest_codes(t):
    """(codes, max|t|) of rows t (float64): round-half-even(127 t / max|t|), decided
    by whole comparisons.  254 |t| is exact for a t of at most 45 bits, and for the
    products of two 16-bit values a quotient that is no tie lies 2^-24 from one at
    least.  Gated values are off by some 2^-52: theirs has a tie where its gate is
    that of the largest value; what lies within 2^-40 of a tie counts as one."""
    t = np.asarray(t, np.float64)
    top = np.abs(t).max(axis=1, keepdims=True)
    two = np.where(top == 0, 1.0, 2 * top)
    over = 254 * np.abs(t) + top
    k = np.floor(over / two + 2.0 ** -40)
    k -= (np.abs(k * two - over) <= two * 2.0 ** -40) & (k % 2 == 1)
    return (k * np.sign(t)).astype(np.int8), top[:, 0]


def add(x, residual):
    """x + residual rounded once to their type: the sum of two 16-bit values in
    float64, rounded through fp32 (24 >= 2 * 11 + 2 bits: rounding twice changes
    nothing)."""
    return (x.to(torch.float64) + residual.to(torch.float64)).to(torch.float32).to(x.dtype)


def norm(x, weight, residual, eps):
    """(values float64, codes, scales float64, total)."""
    h = x if residual is None else add(x, residual)
    v, w = f64(h), f64(weight)
    r = 1 / np.sqrt(np.square(v).mean(axis=1) + np.float64(np.float32(eps)))
    t = v * w
    codes, top = nearest_codes(t)
    return t * r[:, None], codes, np.where(top == 0, 1.0, top * r / 127), h


def gated(x, gate):
    v = f64(x)
    if gate is None:
        return v
    g = f64(gate)
    e = np.exp(-np.abs(g))
    return v * g * np.where(g < 0, e, 1.0) / (1 + e)


def rows(x, gate):
    """(codes, scales float64)."""
    codes, top = nearest_codes(gated(x, gate))
    return codes, np.where(top == 0, 1.0, top / 127)


def product(a, a_scales, w, w_scales, bias, dtype):
    """Y bit for bit: the exact sum, then fp32 steps, each rounded by itself.
    float64 products of int8 are exact below 2^53."""
    acc = a.astype(np.float64) @ w.astype(np.float64).T
    y = acc.astype(np.float32) * a_scales.astype(np.float32)[:, None]
    y = y * w_scales.astype(np.float32)
    if bias is not None:
        y = y + bias.to(torch.float32).numpy()
    with np.errstate(over="ignore"):
        return torch.from_numpy(y).to(dtype)


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)
