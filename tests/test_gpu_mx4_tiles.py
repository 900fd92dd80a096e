"""GPU tests of every form of the 4-bit product, against the product of the held values in float64.

Sizes are the smallest of a search whose estimated time (the choice in mx4_matmul.hip) takes the form named, each
also with more steps of 128 than its ring of stages holds (3 or 4), or than a wave of the few-rows form goes
through at once (32 by eight waves); odd, so that tiles, panels and steps end inside. Tolerance, s the sum of
|a b| over k: 2 k 2^-24 s for the fp32 sums, and 2^-8 of a bf16 result.
"""
import pytest
import torch

import orthogonalized_momentum_optimizer_amd as om
from test_gpu_mx4_linear import dev

pytestmark = pytest.mark.gpu

SIZES = [
    # few rows: one panel or two of B beside A's panels, and of A beside B's
    (1, 18, 133), (16, 18, 2232), (16, 500, 4282), (18, 1, 131), (21, 16, 2052), (600, 13, 4805),
    (17, 17, 129), (17, 300, 2420), (31, 8000, 4187), (19, 17, 134), (18, 17, 2150), (8001, 32, 4513),
    # 128 x 128: whole, split, split with parts of more steps than the ring's
    (33, 33, 135), (34, 35, 664), (129, 257, 641), (34, 33, 1102), (193, 1376, 2080), (65, 64, 20001),
    # 128 x 256
    (7512, 1040, 131), (1677, 4685, 129), (5431, 1410, 674), (1794, 4425, 2001),
    # 256 x 128
    (7620, 2055, 128), (3210, 4874, 133), (7604, 2087, 659), (6015, 2609, 744),
    # 256 x 256: whole, and split
    (6756, 1187, 4388), (4090, 4003, 5001), (4744, 796, 15967)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_matches_float64(m, n, k):
    g = torch.Generator(device=dev()).manual_seed(m + n + k)
    a, b = (torch.randn(r, k, device=dev(), generator=g) * torch.exp2(
        torch.randint(-4, 5, (r, 1), device=dev(), generator=g).float()) for r in (m, n))
    q, p = om.mx4_quantize(a), om.mx4_quantize(b)
    x, y = q.dequantize(torch.float32).double(), p.dequantize(torch.float32).double()
    want, s = x @ y.t().contiguous(), x.abs() @ y.abs().t().contiguous()
    tol = 2 * k * 2.0 ** -24 * s
    for dtype in (torch.float32, torch.bfloat16):
        got = om.mx4_matmul(q, p, dtype)
        err = (got.double() - want).abs()
        assert got.dtype == dtype and bool((err <= tol + (2.0 ** -8 * want.abs() if dtype is torch.bfloat16 else 0)).all()), \
            float((err / tol).max())
        assert torch.equal(got, om.mx4_matmul(q, p, dtype))


@pytest.mark.parametrize("m,n,k", [(7512, 1040, 674), (7604, 2087, 659), (4090, 4003, 5001), (1030, 500, 2001)])
def test_a_product_of_whole_numbers_is_exact(m, n, k):
    """Codes of whole numbers and scales of 1: sums below 2^24, the same in any order."""
    g = torch.Generator(device=dev()).manual_seed(k)
    a, b = (torch.randint(-4, 5, (r, k), device=dev(), generator=g).float() for r in (m, n))
    for t in (a, b):
        t[:, ::32] = 6.0                          # the scale of every block is 1
    got = om.mx4_matmul(om.mx4_quantize(a), om.mx4_quantize(b), torch.float32)
    assert torch.equal(got.double(), a.double() @ b.double().t().contiguous())
