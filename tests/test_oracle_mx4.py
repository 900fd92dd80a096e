"""The oracle of microscaled 4-bit values against the format's tables, bounds and unbiasedness, and
planted mistakes (no GPU)."""
import numpy as np
import pytest

import oracle.mx4 as mx


def row(values):
    out = np.zeros((1, 32))
    out[0, :len(values)] = values
    return out


def test_grid_ties_and_signs():
    """Every tie goes to the even code, values beside it to their own side; -0 keeps its sign."""
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    want = [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    for t, w in zip(ties, want):
        i = list(mx.VALUES).index(w)
        lo, hi = max(v for v in mx.VALUES if v < t), min(v for v in mx.VALUES if v > t)
        x = row([6.0, t, t * (1 - 1e-9), t * (1 + 1e-9), -t])
        c, s = mx.quantize(x)
        assert s[0, 0] == 127
        assert list(mx.values(c, s)[0, :5]) == [6.0, w, lo, hi, -w]
        assert c[0, 1] == i and c[0, 4] == i + 8
    assert mx.quantize(row([-0.0]))[0][0, 0] == 8


@pytest.mark.parametrize("k", [-127, -126, -20, 0, 60, 125])
def test_scale_is_the_smallest_that_cuts_nothing_off(k):
    unit = 2.0 ** k
    for top, byte in ((6.0, 127), (6.0 * (1 + 2 ** -23), 128), (3.0 * (1 + 2 ** -23), 127), (4.0, 127)):
        assert mx.quantize(row([top * unit]))[1][0, 0] == max(byte + k, 0)
    assert mx.quantize(row([3.0 * unit]))[1][0, 0] == max(126 + k, 0)


def test_edges_of_the_range():
    assert mx.quantize(row([]))[1][0, 0] == 0                    # zeros: the smallest scale
    c, s = mx.quantize(row([2.0 ** -149, 2.0 ** -128, 2.0 ** -129]))
    assert s[0, 0] == 0 and list(c[0, :3]) == [0, 1, 0]
    big = float(np.finfo(np.float32).max)
    c, s = mx.quantize(row([big, -big, 2.0 ** 127]))
    assert s[0, 0] == 253 and list(mx.values(c, s)[0, :3]) == [3 * 2.0 ** 126, -3 * 2.0 ** 126, 2.0 ** 127]
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones((1, 64))
        x[0, 5] = bad
        c, s = mx.quantize(x)
        assert list(s[0]) == [255, 125] and not c[0, :32].any()
        v = mx.values(c, s)[0]
        assert np.isnan(v[:32]).all() and (v[32:] == 1).all()


def test_rounding_is_within_half_a_step_and_stochastic_within_one():
    r = np.random.default_rng(1)
    x = r.normal(size=(50, 320)) * 2.0 ** r.integers(-30, 30, (50, 1))
    for seed, most in ((None, 0.5), (3, 1.0)):
        q = mx.hold(x, seed)
        unit = np.repeat(np.ldexp(1.0, mx.quantize(x)[1].astype(int) - 127), 32, axis=1)
        y = np.abs(x) / unit
        step = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0)) * unit
        assert (np.abs(q - x) <= most * step * (1 + 1e-12)).all()
        assert (np.abs(q) <= 6 * unit).all()


def test_stochastic_rounding_is_unbiased():
    """Over all 65536 values of the bits the mean is the value itself, to half a bit's weight."""
    bits = np.arange(65536).reshape(-1, 32)
    for y in (0.1, 0.3, 1.1, 1.99, 2.7, 3.999, 4.3, 5.9):
        x = np.full((2048, 32), y)
        first = np.concatenate([np.full((2048, 32), 6.0), x], axis=1)   # (a block of its own scale)
        assert (mx.quantize(first, np.concatenate([bits, bits], axis=1))[1][:, 0] == 127).all()
        c, s = mx.quantize(x, bits)
        q = mx.values(c, s)
        unit = 2.0 ** (int(s[0, 0]) - 127)
        h = y / unit
        h = unit * (0.5 if h < 2 else 1 if h < 4 else 2)
        assert abs(q.mean() - y) <= h / 65536 and q.max() - q.min() <= h


@pytest.mark.parametrize("seed", [0, 7, 2 ** 63 + 5])
def test_rounding_bits_are_uniform_and_uncorrelated(seed):
    n = 512
    u = (mx.rounding_bits(n, n, seed) + 0.5) / 65536 - 0.5
    m, sd = n * n, 1 / np.sqrt(12.0)
    assert abs(u.mean()) <= 5 * sd / np.sqrt(m)
    assert abs(u.var() - 1 / 12) <= 5 * np.sqrt(1 / 180 / m)
    for a, b in ((u[:, :-1], u[:, 1:]), (u[:-1], u[1:]), (u[:, :-2], u[:, 2:]), (u, u.T)):
        assert abs(np.mean(a * b)) <= 5 / 12 / np.sqrt(m / 2)
    other = (mx.rounding_bits(n, n, seed + 1) + 0.5) / 65536 - 0.5
    assert abs(np.mean(u * other)) <= 5 / 12 / np.sqrt(m)


def test_linear_is_exact_where_nothing_is_rounded():
    r = np.random.default_rng(2)
    x, w, dy = (r.choice([-1.5, -1.0, -0.5, 0.5, 1.0, 3.0], s) for s in ((8, 40), (6, 40), (8, 6)))
    y, dx, dw = mx.linear(x, w, dy)
    assert np.array_equal(y, x @ w.T) and np.array_equal(dx, dy @ w) and np.array_equal(dw, dy.T @ x)


@pytest.mark.parametrize("mistake", ["floor_scale", "away", "truncate", "sign", "no_half_step"])
def test_planted_mistakes_differ(mistake):
    """A quantiser with one of these mistakes is told from the oracle by the inputs of the GPU tests."""
    r = np.random.default_rng(4)
    x = r.normal(size=(16, 64))
    x[:, :7] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    x[:, 7] = 6.0
    good = mx.values(*mx.quantize(x))
    b = x.reshape(16, 2, 32)
    k = np.ceil(np.log2(np.abs(b).max(axis=2) / 6.0))
    if mistake == "floor_scale":
        k = np.floor(np.log2(np.abs(b).max(axis=2))) - 2
    y = np.abs(b) / np.exp2(k)[:, :, None]
    step = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
    if mistake == "no_half_step":
        step = np.where(y < 1, 1.0, step)
    n = {"away": np.floor(y / step + 0.5), "truncate": np.floor(y / step)}.get(mistake, np.rint(y / step))
    q = np.minimum(n * step, 6) * np.exp2(k)[:, :, None] * (1 if mistake == "sign" else np.sign(b))
    assert not np.array_equal(q.reshape(16, 64), good)
