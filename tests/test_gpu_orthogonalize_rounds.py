"""GPU tests of many Newton-Schulz rounds on stacks without full rank.

Rounds on a matrix X in fp32 lift what rounding leaves where X has nothing, by a^n over n rounds, up to
where it is as large as the rest. The operator promises no more than that, and so is measured against
it: fp32 rounds on X itself, formed here on the CPU, are off from the float64 oracle by some Frobenius norm;
the operator may be by four times that (a few roundings in place of one, in each round or each pass)
and, for bf16, 2^-8 of the result. However many the rounds, no singular value passes what they can
make of any in [0, 1.2] (convergent rounds: [0, 1]; 1% for the rounding to bf16, and what the noise adds to those that are there).
"""
import numpy as np
import pytest
import torch

import orthogonalized_momentum_optimizer_amd as om
from test_gpu_orthogonalize import ABC, DT, check, dev, f32, f64, gradients

pytestmark = pytest.mark.gpu

TWO, CUBIC = (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)
SIZES = [(16, 500), (30, 40), (64, 768), (100, 300), (20, 1400)]
KINDS = ["rank1", "rank8", "sums", "same"]


def low_rank(kind, s, l, dtype, seed):
    r = np.random.default_rng(seed)
    if kind == "sums":                            # whole numbers: sums of rows are exact in bf16
        b = r.integers(-8, 9, (s // 2, l))
        x = np.concatenate([b, b[::-1] + np.roll(b, 1, 0)])
    elif kind == "same":                          # every row four times
        x = r.normal(size=(s // 4 + 1, l))[np.arange(s) // 4]
    else:
        k = int(kind[4:])
        u, _ = np.linalg.qr(r.normal(size=(s, k)))
        v, _ = np.linalg.qr(r.normal(size=(l, k)))
        x = u @ np.diag(np.linspace(1, 0.3, k)) @ v.T
    return torch.tensor(x, dtype=torch.float64).to(DT[dtype]).to(dev())


def rounds_on_x(x, rounds, dtype):
    x = (x / (np.sqrt(np.sum(x * x)) + f32(1e-7))).astype(dtype)
    for abc in rounds:
        a, b, c = (dtype(np.float32(v)) for v in abc)
        A = x @ x.T
        x = a * x + (b * A + c * (A @ A)) @ x
    return x


def bounded(got, abc):
    o = f64(got)
    assert np.isfinite(o).all()
    a, b, c = abc
    sigma = np.linspace(0, 1.2 if abc is ABC else 1.0, 20001)
    most = np.abs(sigma * (a + b * sigma ** 2 + c * sigma ** 4)).max()
    assert np.linalg.norm(o, 2) <= 1.01 * most, np.linalg.norm(o, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("abc", [ABC, TWO, CUBIC])
@pytest.mark.parametrize("steps", [8, 9, 12, 20, 64])
@pytest.mark.parametrize("kind", KINDS)
def test_low_rank(kind, steps, abc, dtype):
    for s, l in SIZES:
        x = low_rank(kind, s, l, dtype, s + steps)
        for m in (x, x.t()):
            out = om.orthogonalize(m, steps=steps, abc=abc)
            assert out.stride() == m.stride()
            bounded(out, abc)
        if steps > 20 or kind == "same":
            continue                              # (equal rows stay equal in the rounds on X: no noise to compare with)
        g = f64(x)
        want = rounds_on_x(g, [abc] * steps, np.float64)
        tol = 4 * np.linalg.norm(rounds_on_x(g, [abc] * steps, np.float32) - want)
        if dtype == "bf16":
            tol += 2.0 ** -8 * np.linalg.norm(want)
        err = np.linalg.norm(f64(out).T - want)
        assert err <= tol, (s, l, err, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("steps", [9, 16])
def test_several_passes_agree_with_the_oracle(steps, dtype):
    """Full rank, a convergent round, and every way a stack can lie; eps counts in the first pass only."""
    for shape in ((3, 40, 300), (3, 300, 40), (2, 100, 130), (2, 90, 2000), (70, 12, 20)):
        x = gradients(shape, dtype, steps)
        out = om.orthogonalize(x, steps=steps, abc=TWO, eps=1e-2)
        check(f64(x[0]), out[0], [TWO] * steps, eps=1e-2)
        check(f64(x[-1]), out[-1], [TWO] * steps, eps=1e-2)
    w = gradients((50, 3 * 40), dtype, 1)
    heads = w.view(50, 3, 40).transpose(0, 1)
    long = [(30.0, 0.0, 0.0), (0.03, 0.0, 0.0)] + [TWO] * 16        # two passes
    out = om.orthogonalize(heads, steps=18, schedule=long)
    assert out.stride() == heads.stride()
    buf = torch.full((3, 50, 60), 7.0, device=dev(), dtype=w.dtype)
    assert torch.equal(om.orthogonalize(heads, steps=18, schedule=long, out=buf[:, :, 9:49]), out)
    assert (buf[:, :, :9] == 7).all() and (buf[:, :, 49:] == 7).all()
    om.orthogonalize(heads, steps=18, schedule=long, out=heads)
    assert torch.equal(heads, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zeros_nan_and_range_over_several_passes(dtype):
    for s, l in ((12, 60), (50, 100), (100, 140)):
        x = gradients((6, s, l), dtype, s, scale=1.0)
        x[5] *= 1e18
        want = om.orthogonalize(x, steps=20)
        x[1] = 0
        x[2, 3, 7] = float("nan")
        x[3, s - 1, l - 1] = float("inf")
        out = om.orthogonalize(x, steps=20)
        assert not out[1].any() and out[2].isnan().all() and out[3].isnan().all()
        assert all(torch.equal(out[i], want[i]) for i in (0, 4, 5))
        bounded(out[0], ABC), bounded(out[5], ABC)


def test_several_passes_in_a_graph():
    x = gradients((5, 60, 200), "bf16", 3)
    y = gradients((5, 100, 200), "f32", 4)
    step = lambda: (om.orthogonalize(x, steps=12), om.orthogonalize(y, steps=12))  # noqa: E731
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for k in range(4):
        x.copy_(gradients((5, 60, 200), "bf16", 30 + k))
        y.copy_(gradients((5, 100, 200), "f32", 40 + k))
        g.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step())), k
