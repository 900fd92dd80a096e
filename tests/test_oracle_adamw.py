"""The AdamW oracle against its pins (no GPU): PyTorch's AdamW in float64, PyTorch's e4m3
conversion, the unbiasedness and bounds of the 8-bit form, and planted mistakes."""
import numpy as np
import pytest
import torch

import adamw_ref
import oracle.adamw as oa


def test_step_matches_torch_adamw_in_float64():
    r = np.random.default_rng(1)
    p0 = r.normal(0, 1, 500)
    P = torch.nn.Parameter(torch.tensor(p0))
    opt = torch.optim.AdamW([P], lr=1e-2, betas=(0.8, 0.97), eps=1e-6, weight_decay=0.3,
                            foreach=False)
    p, m, v = p0, np.zeros(500), np.zeros(500)
    for t in range(1, 8):
        g = r.normal(0, 1, 500)
        P.grad = torch.tensor(g)
        opt.step()
        p, m, v = oa.adamw_step(p, 0.5 * g, m, v, t, 1e-2, 0.8, 0.97, 1e-6, 0.3, grad_scale=2.0)
        assert np.allclose(p, P.detach().numpy(), rtol=1e-12, atol=1e-13)
        assert np.allclose(v, opt.state[P]["exp_avg_sq"].numpy(), rtol=1e-12, atol=0)


def test_e4m3_grid_and_rounding_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    values = adamw_ref.e4m3_values(codes).astype(np.float64)
    values = values[np.isfinite(values)]
    assert np.array_equal(oa.e4m3(values), values)
    pos = np.unique(np.abs(values))
    mid = (pos[1:] + pos[:-1]) / 2                       # exact ties, and just beside them
    x = np.concatenate([mid, mid * (1 + 2 ** -20), mid * (1 - 2 ** -20)])
    x = np.concatenate([x, -x])
    assert np.array_equal(oa.e4m3(x), adamw_ref.e4m3_values(adamw_ref.e4m3_codes(x)).astype(np.float64))
    assert np.array_equal(oa.e4m3([453.0, -453.0, 1e9]), [448.0, -448.0, 448.0])


def test_stochastic_rounding_is_unbiased():
    """Over all 65536 values of the bits the mean is the value itself, to half a bit's weight."""
    up = (np.arange(65536) + 0.5) / 65536
    for y in (300.3, 17.9, 1.0, 2 ** -6 + 1e-4, 0.011, 2 ** -9, 3e-4, 447.9, 0.0):
        q = oa.e4m3_step(y)
        got = oa.e4m3(np.full(65536, y), up)
        assert abs(got.mean() - y) <= q / 65536
        assert got.max() - got.min() <= q


@pytest.mark.parametrize("seed,step", [(0, 1), (7, 1), (7, 2), (2 ** 63 + 5, 10 ** 6)])
def test_rounding_bits_are_uniform_and_uncorrelated(seed, step):
    n = 1 << 18
    u = (oa.rounding_bits(np.arange(n), seed, step) + 0.5) / 65536 - 0.5
    sd = 1 / np.sqrt(12.0)
    assert abs(u.mean()) <= 5 * sd / np.sqrt(n)
    assert abs(u.var() - 1 / 12) <= 5 * np.sqrt(1 / 180 / n)
    for lag in (1, 2, 3, 16, 256):
        assert abs(np.mean(u[:-lag] * u[lag:])) <= 5 / 12 / np.sqrt(n - lag)
    other = (oa.rounding_bits(np.arange(n), seed, step + 1) + 0.5) / 65536 - 0.5
    assert abs(np.mean(u * other)) <= 5 / 12 / np.sqrt(n)
    far = (oa.rounding_bits(np.arange(n) + 2 ** 33, seed, step) + 0.5) / 65536 - 0.5
    assert abs(np.mean(u * far)) <= 5 / 12 / np.sqrt(n)


def test_block_scale_is_the_smallest():
    r = np.random.default_rng(2)
    x = r.normal(0, 1, (300, 256)) * 10.0 ** r.uniform(-30, 30, (300, 1))
    s = oa.block_scale(x)
    top = np.abs(x).max(1)
    assert np.all(top <= oa.TOP * s) and np.all(top > oa.TOP * s / 2)
    assert np.array_equal(oa.block_scale(np.zeros((2, 256))), [2.0 ** -127] * 2)
    edge = np.zeros((2, 256))
    edge[:, 3] = oa.TOP * 2.0 ** 5 * np.array([1, 1 + 2 ** -40])
    assert np.array_equal(oa.block_scale(edge), [2.0 ** 5, 2.0 ** 6])
    tiny = np.zeros((1, 256))
    tiny[0, 0] = 2.0 ** -140                              # below TOP 2^-127: the lowest scale
    assert oa.block_scale(tiny)[0] == 2.0 ** -127


@pytest.mark.parametrize("stochastic", [False, True])
def test_float32_evaluation_stays_near_the_float64_values(stochastic):
    """The fp32 evaluation that GPU bytes are compared with, against the float64 definition:
    m within half a step of the format, r within one (half without the random bits)."""
    r = np.random.default_rng(3)
    n = 5000
    g = (r.normal(0, 1, n) * 10.0 ** r.uniform(-6, 0, n)).astype(np.float32)
    mc, ms = np.zeros(n, np.uint8), np.zeros(20, np.uint8)
    rc, rs = mc.copy(), ms.copy()
    for t in range(1, 6):
        m0 = oa.held(adamw_ref.e4m3_values(adamw_ref.rows(mc, np.uint8)), adamw_ref.scale_values(ms), n)
        r0 = oa.held(adamw_ref.e4m3_values(adamw_ref.rows(rc, np.uint8)), adamw_ref.scale_values(rs), n)
        b1, b2 = float(np.float32(0.9)), float(np.float32(0.99))
        _, m, v = oa.adamw_step(np.zeros(n), g, m0, r0 ** 2, t, 0.0, b1, b2, 1e-8)
        mc, ms, rc, rs, _, _ = adamw_ref.step_codes(g, mc, ms, rc, rs, 0.9, 0.99, 11, t, stochastic)
        for x, c, s, share in ((m, mc, ms, 0.5), (np.sqrt(v), rc, rs, 1.0 if stochastic else 0.5)):
            sv = np.repeat(adamw_ref.scale_values(s).astype(np.float64), 256)[:n]
            y = adamw_ref.e4m3_values(c) * sv
            step = np.maximum(np.abs(x) / 8, 2.0 ** -9 * sv)   # at most: a step is 2^-3 of a value
            assert np.all(np.abs(y - x) <= (share + 1e-5) * step + 2.0 ** -9 * sv * (share < 1) * (x > 0) / 2)
        assert np.array_equal(rc == 0, v == 0)                 # v dies only where it is zero
        g = (r.normal(0, 1, n) * np.abs(g)).astype(np.float32)


def test_direction_stays_bounded_where_gradients_stop():
    """An element whose gradient becomes zero in a block whose others go on: m and r shrink to
    the bottom of their formats, where r has a floor and m does not, so |u| stays bounded by the
    ratio of the largest m to the largest r (itself at most 7.3 for these betas) times the
    formats' roundings."""
    r = np.random.default_rng(4)
    n, t = 256, 0
    mc, ms, rc, rs = np.zeros(n, np.uint8), np.zeros(1, np.uint8), np.zeros(n, np.uint8), np.zeros(1, np.uint8)
    live = np.arange(n) % 2 == 0
    for t in range(1, 200):
        g = r.normal(0, 1, n) * np.where(live | (t < 20), 1.0, 0.0)
        mc, ms, rc, rs, m, rr = adamw_ref.step_codes(g, mc, ms, rc, rs, 0.9, 0.999, 0, t, True)
        bc = (1 - 0.9 ** t) / np.sqrt(1 - 0.999 ** t)
        ok = rr > 0
        assert np.all(np.abs(m[ok]) / rr[ok] / bc <= 7.3 * (1 + 2 ** -4) / (1 - 2 ** -3) / bc + 1)


def test_grad_norm_oracle():
    gs = [np.array([3.0, 4.0]), np.zeros(0), np.array([12.0])]
    norm, scale, norms = oa.grad_norm(gs, 6.5)
    assert norm == 13.0 and scale == 0.5 and list(norms) == [5.0, 0.0, 12.0]
    assert oa.grad_norm(gs)[1] == 1.0 and oa.grad_norm(gs, 13.0)[1] == 1.0
    assert np.isnan(oa.grad_norm([np.array([np.inf])], 1.0)[1])


MISTAKES = {
    "no_floor": lambda x, up=None, floor=False: ORIGINAL_HOLD(x, up, False),
    "truncated": lambda x, up=None, floor=False: ORIGINAL_HOLD(
        x, np.zeros(np.asarray(x).size), floor),
}
ORIGINAL_HOLD = oa.hold


@pytest.mark.parametrize("mistake", sorted(MISTAKES))
def test_planted_mistakes_show(mistake):
    """hold() with a mistake differs from the fp32 evaluation where the right one agrees."""
    r = np.random.default_rng(5)
    g = np.abs(r.normal(0, 1, 512) * 10.0 ** r.uniform(-8, 0, 512)).astype(np.float32)
    z8, zs = np.zeros(512, np.uint8), np.zeros(2, np.uint8)
    mc, _, rc, _, m, rr = adamw_ref.step_codes(g, z8, zs, z8, zs, 0.9, 0.99, 0, 1, False)
    assert np.array_equal(oa.hold(rr, floor=True)[0].reshape(-1), adamw_ref.e4m3_values(rc))
    assert np.array_equal(oa.hold(m)[0].reshape(-1), adamw_ref.e4m3_values(mc))
    assert not np.array_equal(MISTAKES[mistake](rr, floor=True)[0].reshape(-1),
                              adamw_ref.e4m3_values(rc))


def test_square_of_the_largest_held_root_is_finite():
    """r as the next step squares it: the largest code times the largest scale that fp32's range
    of v calls for, 2^64, has no fp32 square, and the one below it has."""
    top = np.sqrt(np.finfo(np.float32).max)              # of a v at fp32's end
    for x in (top, 250.0 * 2.0 ** 56, 248.0 * 2.0 ** 56, oa.ROOT_TOP):
        r = np.full(256, 1.0)
        r[3] = x
        for up in (None, np.full(256, 1 - 2.0 ** -17)):
            y, s = oa.hold(r, up, floor=True)
            assert s[0] == 2.0 ** 56 and y[0, 3] * s[0] == oa.ROOT_TOP
    with np.errstate(over="ignore"):
        assert np.isfinite(np.float32(oa.ROOT_TOP) ** 2) and np.isinf(np.float32(2.0 ** 64) ** 2)


def test_largest_held_mean_is_finite():
    """Beside a scale of 2^120 the code above 240 stands for 2^128, which fp32 does not hold."""
    top = float(np.finfo(np.float32).max)
    x = np.full(256, 1e38)
    x[:4] = top, -top, 249.0 * 2.0 ** 120, 238.0 * 2.0 ** 120
    y, s = oa.hold(x)
    assert s[0] == 2.0 ** 120
    assert np.array_equal(y[0, :4] * s[0], np.array([1, -1, 1, 1]) * oa.MEAN_TOP)
    with np.errstate(over="ignore"):
        assert np.isfinite(np.float32(oa.MEAN_TOP)) and np.isinf(np.float32(2.0 ** 128))
