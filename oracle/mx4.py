"""Float64 reference of microscaled 4-bit values and their product.

TEST INFRASTRUCTURE ONLY (see the package docstring). Pure numpy in float64.

Rows in blocks of 32 (the OCP microscaling formats' MXFP4: e2m1 values under an e8m0 scale): the
scale is the smallest 2^k, k >= -127, with max |x| <= 6 2^k, and a value becomes the multiple of the
grid's step around |x| / 2^k (1/2 below 2, 1 below 4, 2 up to 6) that is nearest, ties to the even
code, or stochastically step * floor(|x| / (2^k step) + (b + 1/2) / 65536) with 16 random bits b.
"""
from __future__ import annotations

import numpy as np

from .adamw import mix32
from .cautious_adam import _f64

BLOCK = 32
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rounding_bits(rows: int, cols: int, seed: int):
    """The 16 bits of each place: columns 2j and 2j + 1 of row i share mix(j ^ mix(i ^ key))."""
    z = seed % 2 ** 64
    for _ in range(2):
        z = (z ^ (z >> 32)) * 0xE9F8AC216EBC06F5 % 2 ** 64
    key = np.uint64((z ^ (z >> 32)) % 2 ** 32)
    row = mix32(np.arange(rows, dtype=np.uint64) ^ key)[:, None]
    col = np.arange(cols, dtype=np.uint64)[None]
    h = mix32((col >> np.uint64(1)) ^ row)
    return np.where(col % np.uint64(2) == 1, h >> np.uint64(16), h & np.uint64(0xFFFF)).astype(np.int64)


def quantize(x, bits=None):
    """(codes, scale bytes) of a 2-D x: one code (0..15) a value, in rows of whole blocks, and one
    byte a block."""
    x = _f64(x)
    rows, cols = x.shape
    b = np.zeros((rows, -(-cols // BLOCK) * BLOCK))
    b[:, :cols] = x
    b = b.reshape(rows, -1, BLOCK)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    top = np.abs(b).max(axis=2, initial=0.0)
    mant, e = np.frexp(top / 6.0)                # top/6 = mant 2^e, mant in [1/2, 1)
    k = np.maximum(np.where(top > 0, e - (mant == 0.5), -127), -127)
    y = np.abs(b) * np.ldexp(1.0, -k)[:, :, None]
    step = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
    if bits is None:
        q = np.rint(y / step) * step
    else:
        u = np.zeros((rows, b.shape[1] * BLOCK))
        u[:, :cols] = (bits + 0.5) / 65536.0
        q = np.floor(y / step + u.reshape(b.shape)) * step
    q = np.where(k[:, :, None] == 126, np.minimum(q, 3.0), q)      # 4 * 2^126 is beyond fp32
    codes = np.searchsorted(VALUES, q) + 8 * np.signbit(b)
    codes = np.where(bad[:, :, None], 0, codes).reshape(rows, -1)
    return codes.astype(np.uint8), np.where(bad, 255, k + 127).astype(np.uint8)


def values(codes, scales):
    """What codes (one a value) and scale bytes stand for."""
    table = np.concatenate([VALUES, -VALUES])
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return table[codes] * np.repeat(s, BLOCK, axis=1)


def hold(x, seed=None):
    """The values that x's rows are held as; ``seed``: stochastically."""
    x = _f64(x)
    bits = None if seed is None else rounding_bits(*x.shape, seed)
    return values(*quantize(x, bits))[:, :x.shape[1]]


def linear(x, w, dy, seed=None):
    """(y, dx, dw) of a linear layer over held values; ``seed``: of the gradient's rounding."""
    x, w, dy = _f64(x), _f64(w), _f64(dy)
    return (hold(x) @ hold(w).T, hold(dy, seed) @ hold(w.T).T, hold(dy.T, seed) @ hold(x.T).T)
