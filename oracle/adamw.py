"""Float64 reference of the AdamW step, its 8-bit states and the gradient norm.

TEST INFRASTRUCTURE ONLY (see the package docstring). Pure numpy in float64.

AdamW (Loshchilov and Hutter 2019, "Decoupled Weight Decay Regularization"), per element, with
g the gradient times its scale and t >= 1 the index of the step:

    m <- b1 m + (1 - b1) g;   v <- b2 v + (1 - b2) g^2
    p <- p - lr ((m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps) + wd p)

The 8-bit form holds m and r = sqrt(v) of each block of 256 elements in e4m3 (the OCP 8-bit
floating point format: 4 exponent bits of bias 7, 3 mantissa bits, subnormals, largest 448) times
a power of two.
"""
from __future__ import annotations

import numpy as np

from .cautious_adam import _f64, adam_direction, adam_moments

BLOCK = 256
TOP = 256.0 * (1.0 + 0x629146 / 2.0 ** 23)   # a block's largest value, in units of its scale
MEAN_TOP = 240.0 * 2.0 ** 120                # the largest |m| held: the last code that fp32 holds
ROOT_TOP = 240.0 * 2.0 ** 56                 # the largest r held: the last code whose square fp32 holds


def adamw_step(p, g, m, v, t: int, lr: float, beta1: float, beta2: float, eps: float,
               weight_decay: float = 0.0, grad_scale: float = 1.0):
    """One step on one tensor. Returns (p', m', v') as float64 arrays of p's shape."""
    if t < 1:
        raise ValueError("t counts from 1")
    p, g, m, v = _f64(p), _f64(g) * grad_scale, _f64(m), _f64(v)
    m, v = adam_moments(m, v, g, beta1, beta2)
    return p - lr * (adam_direction(m, v, t, beta1, beta2, eps) + weight_decay * p), m, v


def e4m3_step(y):
    """The distance between neighbouring e4m3 values around y (|y| <= 448)."""
    _, e = np.frexp(np.maximum(np.abs(_f64(y)), 2.0 ** -6))
    return np.ldexp(1.0, e - 4)


def e4m3(y, up=None):
    """y on the e4m3 grid: to nearest even, or for y >= 0 with up in (0, 1) cut after adding up
    steps. |y| beyond 448 becomes 448."""
    y = np.clip(_f64(y), -448.0, 448.0)
    q = e4m3_step(y)
    return (np.rint(y / q) if up is None else np.floor(y / q + up)) * q


def blocks_of(x):
    """x flattened to rows of 256, the last one filled with zeros."""
    x = _f64(x).reshape(-1)
    return np.concatenate([x, np.zeros(-x.size % BLOCK)]).reshape(-1, BLOCK)


def block_scale(x):
    """The power of two of each row: the smallest from 2^-127 on with max |x| <= TOP times it."""
    top = np.abs(x).max(axis=1, initial=0.0)
    mant, e = np.frexp(top / TOP)                # top/TOP = mant 2^e, mant in [1/2, 1)
    return np.ldexp(1.0, np.maximum(np.where(top > 0, e - (mant == 0.5), -127), -127))


def hold(x, up=None, floor=False):
    """The values x (any shape; fp32's finite ones) is held as: (codes' values, scales), rows of
    256. ``floor``: x is r."""
    b = blocks_of(x)
    s = block_scale(b)
    b = np.minimum(b, ROOT_TOP) if floor else np.clip(b, -MEAN_TOP, MEAN_TOP)
    if up is not None:
        up = blocks_of(up)
    y = e4m3(b / s[:, None], up)
    if floor:
        y = np.where(b > 0, np.maximum(y, 2.0 ** -9), y)
    return y, s


def held(codes, scales, n: int):
    """The first n values that codes and scales stand for."""
    return (_f64(codes).reshape(-1, BLOCK) * _f64(scales)[:, None]).reshape(-1)[:n]


def mix32(x):
    x = np.asarray(x, dtype=np.uint64)
    m = np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0xEB26D985)) & m
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x4A08C6ED)) & m
    return x ^ (x >> np.uint64(16))


def rounding_bits(index, seed: int, step: int):
    """The 16 bits of each element index of a tensor."""
    z = (seed + step * 0x1493FA689CA113AD) % 2 ** 64
    for _ in range(2):
        z = (z ^ (z >> 32)) * 0xE9F8AC216EBC06F5 % 2 ** 64
    key = np.uint64((z ^ (z >> 32)) % 2 ** 32)
    index = np.asarray(index, dtype=np.uint64)
    pair = index >> np.uint64(1)
    low, high = pair & np.uint64(0xFFFFFFFF), pair >> np.uint64(32)
    h = mix32(low ^ key ^ ((high * np.uint64(0xEB26D985)) & np.uint64(0xFFFFFFFF)))
    return np.where(index % np.uint64(2) == 1, h >> np.uint64(16), h & np.uint64(0xFFFF)).astype(np.int64)


def grad_norm(grads, max_norm: float = np.inf):
    """(norm, scale, norms) of a list of gradients."""
    norms = np.array([np.sqrt(np.sum(_f64(g) ** 2)) for g in grads])
    norm = np.sqrt(np.sum(norms ** 2))
    if not np.isfinite(norm):
        return norm, np.nan, norms
    return norm, (max_norm / norm if norm > max_norm else 1.0), norms
