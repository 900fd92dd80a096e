"""The 8-bit AdamW step evaluated operation by operation in numpy's float32 (each operation
rounded once, to nearest even), as include/adamw.h promises the stored bytes to be formed."""
import numpy as np
import torch

import oracle.adamw as oa

F = np.float32


def f32(x):
    return np.asarray(x, dtype=np.float32)


def e4m3_values(codes):
    return torch.from_numpy(np.ascontiguousarray(codes, np.uint8)).view(torch.float8_e4m3fn).float().numpy()


def e4m3_codes(values):
    """Nearest-even codes of float32 values (of |x| < 464)."""
    t = torch.from_numpy(np.ascontiguousarray(values, np.float32)).to(torch.float8_e4m3fn)
    return t.view(torch.uint8).numpy()


def scale_values(b):
    return np.ldexp(F(1), b.astype(np.int32) - 127).astype(np.float32)


def rows(x, dtype=np.float32):
    x = np.asarray(x, dtype).reshape(-1)
    return np.concatenate([x, np.zeros(-x.size % oa.BLOCK, dtype)]).reshape(-1, oa.BLOCK)


def scale_bytes(x):
    """The smallest b with max |x| <= TOP * 2^(b - 127), by search over all b."""
    top = np.abs(x.astype(np.float64)).max(axis=1)
    limit = oa.TOP * 2.0 ** (np.arange(256) - 127.0)
    return np.minimum(np.searchsorted(limit, top, side="left"), 255).astype(np.uint8)


def step_codes(g, mc, ms, rc, rs, beta1, beta2, seed, step, stochastic, grad_scale=1.0):
    """New (m codes, m scales, r codes, r scales, m, r) from gradients and codes of one tensor of
    n elements; m and r are the float32 values before they are held."""
    n = np.asarray(g).size
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        g = rows(g) * F(grad_scale)
        m = e4m3_values(rows(mc, np.uint8)) * scale_values(ms)[:, None]
        r = e4m3_values(rows(rc, np.uint8)) * scale_values(rs)[:, None]
        b1, b2 = F(beta1), F(beta2)
        m = b1 * m + (F(1) - b1) * g
        v = b2 * (r * r) + (F(1) - b2) * (g * g)
        r = np.sqrt(v)
        top = np.sqrt(np.finfo(np.float32).max)              # an infinite v is held as the largest
        assert m.dtype == r.dtype == np.float32
        mb, rb = scale_bytes(m), scale_bytes(np.minimum(r, top))
        y = m * np.ldexp(F(1), 127 - mb.astype(np.int32)).astype(np.float32)[:, None]
        z = np.minimum(r, top) * np.ldexp(F(1), 127 - rb.astype(np.int32)).astype(np.float32)[:, None]
        w = np.minimum(z, F(448))
        if stochastic:
            bits = oa.rounding_bits(np.arange(w.size), seed, step).reshape(w.shape)
            shift = np.where(w < F(2 ** -6), F(2 ** -6), F(0))
            u = (w + shift).view(np.uint32) + (bits * 16 + 8).astype(np.uint32)
            w = (u & np.uint32(0xFFF00000)).view(np.float32) - shift
        w = np.where(z > 0, np.maximum(w, F(2 ** -9)), z)
        flat = lambda a: a.reshape(-1)[:n]  # noqa: E731
        return flat(e4m3_codes(y)), mb, flat(e4m3_codes(w)), rb, flat(m), flat(r)
