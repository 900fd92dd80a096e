"""GPU tests of microscaled 4-bit quantisation and its product against the float64 oracle.

Codes and scales are compared byte by byte: quantisation has one answer for each value. The product's
tolerance: operands are exact, a product of two has at most 8 bits and sums are fp32. With s the sum
of |a b| over k, an fp32 sum of k terms in any order is off by at most k 2^-24 s (to first order); the
matrix cores may cut instead of rounding, which doubles it. bf16 results are rounded once more, by at
most half a step, 2^-8 of the result. Tests whose partial sums all fit 24 bits
ask for equality.
"""
import numpy as np
import pytest
import torch

import oracle.mx4 as mx
import orthogonalized_momentum_optimizer_amd as om
from orthogonalized_momentum_optimizer_amd import _lib as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev():
    return torch.device("cuda", 0)


def f64(t):
    return t.detach().double().cpu().numpy()


def make(rows, cols, dtype, seed=0):
    """Normal values over twelve binades of row scales, with ties, zeros and whole zero blocks."""
    r = np.random.default_rng(rows * 7919 + cols * 31 + seed)
    x = r.normal(size=(rows, cols)) * 2.0 ** r.integers(-6, 6, (rows, 1))
    ties = r.random((rows, cols)) < 0.1
    x = np.where(ties, r.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.0], (rows, cols)), x)
    x[:, 32:64] *= r.random((rows, 1)) < 0.7
    return torch.tensor(x, dtype=torch.float64).to(DT[dtype]).to(dev())


def unpacked(q):
    """(codes one a value in whole blocks, scale bytes) of an MX4Tensor, from its parts."""
    c, s = (t.cpu().numpy() for t in q.parts())
    blocks = -(-q.cols // 32)
    out = np.zeros((q.rows, blocks * 32), dtype=np.uint8)
    wide = np.stack([c & 15, c >> 4], axis=2).reshape(q.rows, -1)
    out[:, :wide.shape[1]] = wide
    return out, s


def same(q, x, seed=None):
    """q is what the oracle makes of x (numpy)."""
    bits = None if seed is None else mx.rounding_bits(*x.shape, seed)
    c, s = mx.quantize(x, bits)
    got_c, got_s = unpacked(q)
    assert np.array_equal(got_s, s)
    bad = np.argwhere(got_c != c)
    assert not len(bad), (bad[:5], got_c[tuple(bad[0])], c[tuple(bad[0])])


def pads_are_zero(q):
    panels, steps = -(-q.rows // 16), -(-q.cols // 128)
    at = panels * steps * 1024
    c = q.data[:at].view(panels, steps, 16, 64).transpose(1, 2).reshape(panels * 16, -1)
    s = q.data[at:].view(panels, steps, 16, 4).transpose(1, 2).reshape(panels * 16, -1)
    assert not c[q.rows:].any() and not s[q.rows:].any()
    assert not c[:, -(-q.cols // 32) * 16:].any() and not s[:, -(-q.cols // 32):].any()


SIZES = [(1, 1), (1, 31), (1, 32), (3, 33), (15, 127), (16, 128), (17, 129), (64, 96), (65, 7),
         (127, 255), (128, 257), (129, 64), (200, 1000), (1, 5000), (5000, 1), (1013, 769)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_matches_the_oracle(rows, cols, stochastic, dtype):
    x = make(rows, cols, dtype)
    h, seed = f64(x), 12345 if stochastic else None
    how = dict(stochastic=stochastic, seed=12345)
    q = om.mx4_quantize(x, **how)
    assert (q.rows, q.cols, tuple(q.shape)) == (rows, cols, (rows, cols))
    same(q, h, seed)
    a, b = om.mx4_quantize_both(x, **how)
    assert torch.equal(a.data, q.data)
    same(b, h.T, seed)
    t = om.mx4_quantize(x.t(), **how)
    assert torch.equal(t.data, b.data)
    for each in (q, b):
        pads_are_zero(each)
        for dt in DT.values():
            want = mx.values(*unpacked(each))[:, :each.cols]
            assert np.array_equal(f64(each.dequantize(dt)), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_range_and_values_that_are_not_finite(dtype):
    """Scales from 2^-127 to 2^126, subnormals, the top of the range, and NaN or infinity in some
    blocks, which leave the others alone."""
    top = float(torch.finfo(DT[dtype]).max)
    r = np.random.default_rng(5)
    x = r.normal(size=(300, 160)) * 2.0 ** np.linspace(-150, 125, 300)[:, None]
    x[10, :3] = [top, -top, 3.49 * 2.0 ** 126]
    x[11, :3] = [top / 2, 1.0, -1.0]
    x[12, 40], x[13, 0], x[14, 159], x[15, 100] = np.nan, np.inf, -np.inf, np.nan
    x[16:48, 7] = 0.0
    x[20, 7] = np.inf
    x = torch.tensor(x).to(DT[dtype]).to(dev())
    for seed in (None, 9):
        how = dict(stochastic=seed is not None, seed=seed or 0)
        a, b = om.mx4_quantize_both(x, **how)
        same(a, f64(x), seed)
        same(b, f64(x).T, seed)
        for q in (a, b):
            got, want = f64(q.dequantize(torch.float32)), mx.values(*unpacked(q))[:, :q.cols]
            assert np.array_equal(got, want, equal_nan=True)
            assert np.array_equal(f64(q.dequantize(torch.bfloat16)), want, equal_nan=True)


def test_layouts_of_the_source():
    x = make(96, 260, "bf16")
    cut = x[3:70, 5:204]                                    # odd start, rows apart
    same(om.mx4_quantize(cut), f64(cut))
    same(om.mx4_quantize(cut.t()), f64(cut).T)
    a, b = om.mx4_quantize_both(cut.t())
    same(a, f64(cut).T)
    same(b, f64(cut))
    lead = x.view(4, 24, 260)
    q = om.mx4_quantize(lead)
    assert tuple(q.shape) == (4, 24, 260) and torch.equal(q.data, om.mx4_quantize(x).data)
    assert tuple(q.dequantize().shape) == (4, 24, 260)
    one = x[7]
    assert torch.equal(om.mx4_quantize(one).data, om.mx4_quantize(x[7:8]).data)
    assert torch.equal(om.mx4_quantize(x[:, :1]).data, om.mx4_quantize(x[:, :1].contiguous()).data)
    for bad in (x[:, ::2], x.view(4, 24, 260).transpose(0, 1), x[:1].expand(8, 260)):
        with pytest.raises(ValueError):
            om.mx4_quantize(bad)


def test_parts_and_back():
    x = make(37, 77, "f32")
    q = om.mx4_quantize(x)
    codes, scales = q.parts()
    assert tuple(codes.shape) == (37, 39) and tuple(scales.shape) == (37, 3)
    codes[:, 38] |= 0xF0                                    # behind the last value: not read
    again = om.MX4Tensor(codes, scales, 77)
    assert torch.equal(again.data, q.data)
    assert torch.equal(om.MX4Tensor(codes, scales.view(torch.float8_e8m0fnu), 77).data, q.data)


MM = [(1, 1, 1), (1, 16, 32), (2, 17, 33), (5, 300, 129), (16, 64, 128), (17, 100, 500), (33, 257, 640),
      (64, 64, 64), (100, 1000, 777), (128, 128, 256), (129, 127, 1), (250, 260, 1030), (256, 256, 512),
      (257, 511, 384), (300, 2000, 100), (700, 70, 3000), (1000, 900, 2050)]


def check_product(a, b, out, dtype):
    """out against the exact product of the held values a, b (numpy)."""
    want, s = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = 2 * a.shape[1] * 2.0 ** -24 * s + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
    err = np.abs(f64(out) - want)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", MM)
def test_matmul_matches_the_oracle(m, n, k, dtype):
    a, b = make(m, k, "f32", 1), make(n, k, "f32", 2)
    qa, qb = om.mx4_quantize(a), om.mx4_quantize(b)
    out = om.mx4_matmul(qa, qb, out_dtype=DT[dtype])
    assert out.dtype == DT[dtype] and tuple(out.shape) == (m, n)
    check_product(mx.hold(f64(a)), mx.hold(f64(b)), out, dtype)
    assert torch.equal(out, om.mx4_matmul(qa, qb, out_dtype=DT[dtype]))


@pytest.mark.parametrize("m,n,k", [(3, 200, 5000), (130, 140, 9000), (513, 770, 260)])
def test_matmul_is_exact_on_whole_numbers(m, n, k):
    """Values 0, +-1/2, +-1 and scales of 1: every partial sum is a multiple of 1/4 below 2^22."""
    r = np.random.default_rng(m)
    a, b = (torch.tensor(r.choice([0, 0.5, -0.5, 1, -1, 4.0], (s, k)), dtype=torch.float32, device=dev())
            for s in (m, n))
    a[:, ::32], b[:, ::32] = 4.0, 4.0
    out = om.mx4_matmul(om.mx4_quantize(a), om.mx4_quantize(b), out_dtype=torch.float32)
    assert np.array_equal(f64(out), f64(a) @ f64(b).T)


def test_matmul_positions():
    """One value in either operand at a time lands where it belongs, at every place of a tile."""
    m, n, k = 300, 290, 300
    r = np.random.default_rng(0)
    for _ in range(4):
        a, b = torch.zeros(m, k), torch.zeros(n, k)
        cols = torch.tensor(r.permutation(k)[:max(m, n)] if k >= max(m, n) else r.integers(0, k, max(m, n)))
        a[torch.arange(m), cols[:m]] = torch.tensor(r.choice([1.0, 2.0, 3.0, -6.0], m), dtype=torch.float32)
        b[torch.arange(n), cols[torch.tensor(r.permutation(m)[:n])]] = 1.5
        a, b = a.to(dev()), b.to(dev())
        out = om.mx4_matmul(om.mx4_quantize(a), om.mx4_quantize(b), out_dtype=torch.float32)
        assert np.array_equal(f64(out), f64(a) @ f64(b).T)


def test_nan_stays_in_its_row_and_column():
    for m, n, k in ((4, 100, 300), (200, 300, 260)):
        a, b = make(m, k, "f32", 3), make(n, k, "f32", 4)
        a[1, 7], b[33, 130] = float("nan"), float("inf")
        out = f64(om.mx4_matmul(om.mx4_quantize(a), om.mx4_quantize(b), out_dtype=torch.float32))
        want = np.zeros((m, n), dtype=bool)
        want[1], want[:, 33] = True, True
        assert np.array_equal(np.isnan(out), want)


def test_empty_sizes():
    e = lambda *s: torch.empty(*s, device=dev())  # noqa: E731
    assert om.mx4_quantize(e(0, 5)).dequantize().shape == (0, 5)
    assert om.mx4_quantize(e(5, 0)).dequantize().shape == (5, 0)
    a, b = om.mx4_quantize_both(e(0, 5))
    assert (a.rows, b.rows, b.cols) == (0, 5, 0)
    out = om.mx4_matmul(om.mx4_quantize(e(5, 0)), om.mx4_quantize(e(7, 0)), torch.float32)
    assert out.shape == (5, 7) and not out.any()
    assert om.mx4_matmul(om.mx4_quantize(e(0, 9)), om.mx4_quantize(e(7, 9))).shape == (0, 7)


def test_leading_dimensions_of_a_product():
    a, b = make(24, 96, "bf16", 5), make(10, 96, "bf16", 6)
    out = om.mx4_matmul(om.mx4_quantize(a.view(2, 12, 96)), om.mx4_quantize(b))
    assert torch.equal(out, om.mx4_matmul(om.mx4_quantize(a), om.mx4_quantize(b)).view(2, 12, 10))
