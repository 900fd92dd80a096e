"""MX4Tensor from the usual layout and back, on the host."""
import pytest
import torch

import orthogonalized_momentum_optimizer_amd as om


@pytest.mark.parametrize("rows,cols", [(0, 0), (0, 5), (3, 0), (1, 1), (17, 129), (16, 128), (33, 300)])
def test_parts_are_the_way_back(rows, cols):
    half, blocks = -(-cols // 2), -(-cols // 32)
    g = torch.Generator().manual_seed(rows * 1000 + cols)
    codes = torch.randint(0, 256, (rows, half + 2), dtype=torch.uint8, generator=g)
    scales = torch.randint(0, 256, (rows, blocks + 1), dtype=torch.uint8, generator=g)
    q = om.MX4Tensor(codes, scales, cols)
    c, s = q.parts()
    want = codes[:, :half].clone()
    if cols % 2:
        want[:, -1] &= 15
    assert q.shape == (rows, cols) and torch.equal(c, want) and torch.equal(s, scales[:, :blocks])
