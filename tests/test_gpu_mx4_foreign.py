"""GPU tests of held values that other programs made: every scale byte beside every code. 2^(b - 127) code,
and NaN where b is 255, whatever the codes; quantisation itself never writes byte 254, nor codes beside 255.
"""
import numpy as np
import pytest
import torch

import orthogonalized_momentum_optimizer_amd as om
from test_gpu_mx4_linear import DT, dev, f64

pytestmark = pytest.mark.gpu

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def tensor(codes, scales, cols):
    """codes: one a value (numpy, an even number of columns)."""
    packed = (codes[:, ::2] | codes[:, 1::2] << 4).astype(np.uint8)
    return om.MX4Tensor(torch.tensor(packed, device=dev()), torch.tensor(scales.astype(np.uint8), device=dev()), cols)


def values(codes, scales):
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return VALUES[codes] * np.repeat(s, 32, axis=1)[:, :codes.shape[1]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_scale_and_code_has_its_value(dtype):
    codes = np.tile(np.arange(32) % 16, (256, 1))
    scales = np.arange(256)[:, None]
    got = tensor(codes, scales, 32).dequantize(DT[dtype])
    want = torch.tensor(values(codes, scales)).to(DT[dtype])       # (beyond the type's range: infinity)
    assert np.array_equal(f64(got), want.double().numpy(), equal_nan=True)
    assert (torch.signbit(got).cpu() | got.isnan().cpu()).equal(torch.signbit(want) | want.isnan())


@pytest.mark.parametrize("m,n", [(1, 40), (40, 1), (20, 300), (300, 20), (150, 200)])
def test_products_of_every_scale(m, n):
    """A block of each pair of scales whose product is 1, and one code beside it: few rows and tiles."""
    r = np.random.default_rng(m)
    blocks = 255
    a, b = (r.integers(0, 16, (rows, 32 * blocks)) for rows in (m, n))
    sa = np.tile(np.arange(blocks), (m, 1))
    sb = np.tile(254 - np.arange(blocks), (n, 1))
    q, p = tensor(a, sa, 32 * blocks), tensor(b, sb, 32 * blocks)
    want = VALUES[a] @ VALUES[b].T                # multiples of 1/4 below 2^19: exact in fp32, in any order
    assert np.array_equal(f64(om.mx4_matmul(q, p, torch.float32)), want)


@pytest.mark.parametrize("m,n", [(1, 40), (40, 1), (20, 300), (300, 20), (150, 200)])
def test_a_nan_scale_is_a_nan_row_of_the_product(m, n):
    r = np.random.default_rng(n)
    cols = 5 * 128 - 32                           # the last step is in part beyond the matrix
    a, b = (r.integers(0, 16, (rows, cols)) for rows in (m, n))
    sa, sb = (r.integers(120, 132, (rows, cols // 32)) for rows in (m, n))
    sa[m - 1, 3] = 255
    sb[n // 2, cols // 32 - 1] = 255
    a[m - 1, 96:128] = 0                          # codes 0 and others
    got = f64(om.mx4_matmul(tensor(a, sa, cols), tensor(b, sb, cols), torch.float32))
    want = values(a, sa) @ values(b, sb).T        # (more bits than a sum in fp32 has)
    nan = np.zeros((m, n), dtype=bool)
    nan[m - 1], nan[:, n // 2] = True, True
    assert np.array_equal(np.isnan(got), nan)
    s = np.abs(np.nan_to_num(values(a, sa))) @ np.abs(np.nan_to_num(values(b, sb))).T
    assert (np.abs(got - want)[~nan] <= 2 * cols * 2.0 ** -24 * s[~nan]).all()
