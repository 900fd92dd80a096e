"""GPU tests of the orthogonalisation of stacks over the range of their types, against the float64
oracle and with the tolerances of test_gpu_orthogonalize.
"""
import numpy as np
import pytest
import torch

import orthogonalized_momentum_optimizer_amd as om
from test_gpu_orthogonalize import ABC, check, dev, f32, f64, gradients, polynomial

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("s,l", [(12, 40), (12, 1100), (20, 50), (30, 1300), (64, 200), (64, 1500), (100, 140),
                                 (100, 700)])
@pytest.mark.parametrize("scale", [1e-37, 1e-22, 1e-18, 1e-15, 1e-13, 1e-10, 1e10, 1e18, 1e20, 1e36])
def test_every_finite_value_is_in_range(scale, s, l, tall, dtype):
    """In one launch, and in three where few matrices are long or the short side is over 64."""
    x = gradients((2, l, s) if tall else (2, s, l), dtype, s + l, scale=scale)
    out = om.orthogonalize(x, eps=0.0)
    for i in range(2):
        check(f64(x[i]), out[i], [ABC] * 5, eps=0.0)
    assert torch.equal(out, om.orthogonalize(x, eps=0.0))
    out = om.orthogonalize(x)
    check(f64(x[1]), out[1], [ABC] * 5)


@pytest.mark.parametrize("s,l", [(20, 3000), (100, 3000)])
def test_pieces_of_other_magnitudes(s, l):
    """A long side whose pieces are summed apart: large, tiny and empty ones. The tiny values are 1e-52 of
    the norm: their results, at most 485 |x| long, lie below every bf16 value (9e-41), and what they add to the
    Gram matrix is 1e-100 of it; so the others are compared with what they are without them."""
    x = gradients((2, s, l), "bf16", l, scale=1.0)
    x[:, :, 600:1200] *= 1e22
    x[:, :, 1200:1800] *= 1e-30
    x[:, :, 1800:2400] = 0
    out = om.orthogonalize(x, eps=0.0)
    assert not out[:, :, 1200:2400].any()
    x[:, :, 1200:1800] = 0
    for i in range(2):
        check(f64(x[i]), out[i], [ABC] * 5, eps=0.0)


@pytest.mark.parametrize("s,l", [(16, 1500), (40, 60), (64, 1500), (100, 140)])
@pytest.mark.parametrize("tall", [False, True])
def test_zeros_nan_and_infinity_stay_in_their_bf16_matrix(s, l, tall):
    x = gradients((5, l, s) if tall else (5, s, l), "bf16", s)
    want = om.orthogonalize(x)
    x[1] = 0
    x[2, 3, 7] = float("nan")
    x[3, -1, -1] = float("-inf")
    out = om.orthogonalize(x)
    assert not out[1].any() and out[2].isnan().all() and out[3].isnan().all()
    assert torch.equal(out[0], want[0]) and torch.equal(out[4], want[4])


def lift(lam, rounds):
    """How far an error of A_0 moves the result: the largest |P(a) - P(b)| / |a - b| sqrt(b) over the
    eigenvalues (the derivative where they meet)."""
    p, dp = polynomial(lam, rounds)
    d = lam[:, None] - lam[None]
    meet = np.abs(d) <= 1e-9 * (lam[:, None] + lam[None]) + 1e-300
    q = np.where(meet, dp[:, None], (p[:, None] - p[None]) / np.where(meet, 1, d))
    return np.abs(q * np.sqrt(lam)[None]).max()


def norm_check(x, got, rounds):
    """A bf16 result in Frobenius norm. As test_gpu_orthogonalize's tolerance, and: the Gram matrix's sums of
    32 in fp32, each off by at most sqrt(31 / 3) 2^-24 |x_i| |x_j| (31 roundings of independent sign, uniform), and
    l / 32 of them independent: A_0 of trace 1 is off by at most 3.3 2^-24 sqrt(32 / l), below 2^-19 / sqrt(l)."""
    rounds = [tuple(f32(v) for v in abc) for abc in rounds]
    s, l = x.shape
    n = x / (np.sqrt(np.sum(x * x)) + f32(1e-7))
    lam, v = np.linalg.eigh(n @ n.T)
    lam = np.maximum(lam, 0)
    want = n
    for a, b, c in rounds:
        A = want @ want.T
        want = a * want + (b * A + c * (A @ A)) @ want
    P = (v * polynomial(lam, rounds)[0]) @ v.T
    tol = 2 * (s + 3) * 2.0 ** -24 * np.linalg.norm(np.abs(P) @ np.abs(n))
    tol += lift(lam, rounds) * 2.0 ** -19 / np.sqrt(l) + 2.0 ** -8 * np.linalg.norm(want)
    err = np.linalg.norm(f64(got) - want)
    assert err <= tol, (err, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_directions_and_low_rank(dtype):
    """Spectra of five decades, eight directions rounded to the type, and rows that stand there many times."""
    r = np.random.default_rng(3)
    for s, l in ((12, 40), (17, 50), (60, 60), (64, 300), (120, 200)):
        u, _ = np.linalg.qr(r.normal(size=(s, s)))
        v, _ = np.linalg.qr(r.normal(size=(l, s)))
        some = np.where(np.arange(s) < 8, 1.0, 0.0)
        for m in (u @ np.diag(np.logspace(0, -5, s)) @ v.T, u @ np.diag(some) @ v.T,
                  r.normal(size=(8, l))[np.arange(s) % 8]):
            x = torch.tensor(m).to(torch.bfloat16 if dtype == "bf16" else torch.float32).to(dev())
            (norm_check if dtype == "bf16" else check)(f64(x), om.orthogonalize(x), [ABC] * 5)


def test_equal_matrices_in_every_batch():
    """More matrices than a launch takes: the last, small batch is summed as the others are. (Small
    directions and eight rounds show a sum's last bits in the result.)"""
    r = np.random.default_rng(4)
    u, _ = np.linalg.qr(r.normal(size=(256, 17, 17)))
    v, _ = np.linalg.qr(r.normal(size=(256, 150, 17)))
    m = torch.tensor(u * np.logspace(0, -5, 17) @ v.swapaxes(1, 2), dtype=torch.float32, device=dev())
    x = m[torch.arange(2 ** 20 + 256, device=dev()) % 256]
    out = om.orthogonalize(x, steps=8)
    assert torch.equal(out[-256:], out[:256]) and torch.equal(out[2 ** 19:2 ** 19 + 256], out[:256])


def test_forward_mode_derivatives_are_refused():
    """Where a backward pass is refused a tangent is not dropped either."""
    from torch.autograd import forward_ad
    x, t = gradients((2, 8, 16), "f32", 1), gradients((2, 8, 16), "f32", 2)
    want = om.orthogonalize(x)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, t)
        for call in (lambda: om.orthogonalize(dual), lambda: om.orthogonalize(x, out=dual),
                     lambda: om.orthogonalize(dual, out=torch.empty_like(x))):
            with pytest.raises(ValueError, match="forward-mode"):
                call()
        assert torch.equal(om.orthogonalize(forward_ad.unpack_dual(dual).primal), want)
