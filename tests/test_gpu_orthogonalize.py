"""GPU tests of the orthogonalisation of stacks of small matrices against the float64 oracle.

Tolerance, per element, with P the polynomial of the Gram matrix (from the oracle, in float64) and x
the normalised matrix, short side as rows:
* the product P x in fp32: P is rounded once, a sum of s terms may be cut instead of rounded, the
  result is rounded: 2 (s + 3) 2^-24 (|P| |x|);
* the Gram matrix and rounds in double: errors of 10 (l + s) 2^-53 in A (||A|| <= 1) change P by at
  most that times D = max |dQ/dlambda| over [0, 1.02], Q the rounds' scalar polynomial, and so an
  element by that times the norm of its column of x;
* bf16: 2^-8 of the result, half a step. (A bf16 stack's Gram matrix is made of fp32 sums of 32 exact
  products, added in double. What those are off by, up to 32 2^-24 |x| |x|^T times D, is not allowed for:
  the bound asked for is the smaller one without it.)
"""
import numpy as np
import pytest
import torch

import oracle
import orthogonalized_momentum_optimizer_amd as om

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ABC = (3.4445, -4.7750, 2.0315)
CASCADE = [(4.0, -7.5, 4.5), (3.9, -6.5, 3.4), (3.5, -5.0, 2.2)]


def dev():
    return torch.device("cuda", 0)


def f64(t):
    return t.detach().double().cpu().numpy()


def f32(x):
    return float(np.float32(x))


def polynomial(lam, rounds):
    """(P, slope) of the rounds at eigenvalues lam of A_0: P with X_r = P X_0, and dP/dlam."""
    p, dp = np.ones_like(lam), np.zeros_like(lam)
    for a, b, c in rounds:
        mu, dmu = p * p * lam, 2 * p * dp * lam + p * p
        q, dq = a + b * mu + c * mu * mu, (b + 2 * c * mu) * dmu
        p, dp = q * p, dq * p + q * dp
    return p, dp


def check(x, got, rounds, eps=1e-7):
    """got against the oracle for one matrix (numpy x; torch got)."""
    rounds = [tuple(f32(v) for v in abc) for abc in rounds]
    g, o = (x, f64(got)) if x.shape[0] <= x.shape[1] else (x.T, f64(got).T)
    s, l = g.shape
    n = g / (np.sqrt(np.sum(g * g)) + f32(eps))
    lam, v = np.linalg.eigh(n @ n.T)
    p, _ = polynomial(np.maximum(lam, 0), rounds)
    P = (v * p) @ v.T
    # (the oracle's rounds on X itself, which lose less than the eigenvectors of A_0)
    want = n
    for a, b, c in rounds:
        A = want @ want.T
        want = a * want + (b * A + c * (A @ A)) @ want
    slope = np.abs(polynomial(np.linspace(0, 1.02, 20001), rounds)[1]).max()
    tol = (2 * (s + 3) * 2.0 ** -24 * (np.abs(P) @ np.abs(n)) +
           10 * (l + s) * 2.0 ** -53 * slope * np.sqrt(np.sum(n * n, axis=0))[None])
    if got.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    err = np.abs(o - want)
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), err.max())


def gradients(shape, dtype, seed, scale=1e-4):
    """Noise and, where there is room, three strong directions in each matrix."""
    r = np.random.default_rng(seed)
    x = r.normal(size=shape)
    k = min(3, shape[-1], shape[-2])
    x += 3 * r.normal(size=shape[:-1] + (k,)) @ r.normal(size=shape[:-2] + (k, shape[-1]))
    return torch.tensor(x * scale).to(DT[dtype]).to(dev())


SIZES = [(1, 1), (1, 7), (2, 2), (3, 100), (5, 5), (8, 1000), (15, 16), (16, 16), (16, 768), (17, 33),
         (31, 64), (32, 32), (32, 500), (33, 129), (48, 100), (63, 65), (64, 64), (64, 768), (64, 1601),
         (65, 66), (80, 333), (100, 100), (127, 300), (128, 128), (128, 1000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("s,l", SIZES)
def test_matches_the_oracle(s, l, tall, dtype):
    x = gradients((3, l, s) if tall else (3, s, l), dtype, s * 1000 + l)
    out = om.orthogonalize(x)
    assert out.shape == x.shape and out.dtype == x.dtype and out.stride() == x.stride()
    for i in range(3):
        check(f64(x[i]), out[i], [ABC] * 5)
    assert torch.equal(out, om.orthogonalize(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rounds", [0, 1, 2, 8])
def test_rounds_and_schedules(rounds, dtype):
    for s, l in ((12, 40), (30, 30), (64, 200), (96, 130)):
        x = gradients((2, s, l), dtype, rounds + s)
        out = om.orthogonalize(x, steps=rounds)
        for i in range(2):
            check(f64(x[i]), out[i], [ABC] * rounds)
    out = om.orthogonalize(x, steps=3, schedule=CASCADE, eps=1e-3)
    for i in range(2):
        check(f64(x[i]), out[i], CASCADE, eps=1e-3)
    out = om.orthogonalize(x, steps=2, abc=(2.0, -1.5, 0.5))
    check(f64(x[0]), out[0], [(2.0, -1.5, 0.5)] * 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_heads_as_they_lie_in_projections(dtype):
    """Rows split by head, columns split by head, and a stack of layers of either."""
    w = gradients((6 * 64, 200), dtype, 1)
    rows = w.view(6, 64, 200)
    out = om.orthogonalize(rows)
    for h in range(6):
        check(f64(rows[h]), out[h], [ABC] * 5)
    w = gradients((300, 5 * 48), dtype, 2)
    cols = w.view(300, 5, 48).transpose(0, 1)
    out = om.orthogonalize(cols)
    assert out.stride() == cols.stride()
    for h in range(5):
        check(f64(cols[h]), out[h], [ABC] * 5)
    w = gradients((3, 90, 4 * 24), dtype, 3)
    both = w.view(3, 90, 4, 24).permute(0, 2, 1, 3)
    out = om.orthogonalize(both)
    for i in range(3):
        for h in range(4):
            check(f64(both[i, h]), out[i, h], [ABC] * 5)
            assert torch.equal(out[i, h], om.orthogonalize(both[i, h]))
    cut = w[:, 3:81, 5:90]                        # rows apart, odd start; a matrix of 78 x 85
    out = om.orthogonalize(cut)
    check(f64(cut[2]), out[2], [ABC] * 5)
    flipped = w[0, :, :17].t()                    # columns contiguous, the short side as rows
    check(f64(flipped), om.orthogonalize(flipped), [ABC] * 5)


def test_out_and_in_place():
    x = gradients((4, 64, 130), "f32", 5)
    want = om.orthogonalize(x)
    buf = torch.full((4, 64, 160), 7.0, device=dev())
    got = om.orthogonalize(x, out=buf[:, :, 9:139])
    assert torch.equal(got, want) and (buf[:, :, :9] == 7).all() and (buf[:, :, 139:] == 7).all()
    assert om.orthogonalize(x, out=x) is x and torch.equal(x, want)
    for tall in (gradients((2, 700, 100), "bf16", 6), gradients((700, 2, 33), "f32", 6).transpose(0, 1)):
        want = om.orthogonalize(tall)
        om.orthogonalize(tall, out=tall)
        assert torch.equal(tall, want)


@pytest.mark.parametrize("scale", [1e-44, 1e-30, 1e-12, 1e12, 1e30, 1e37])
def test_range_of_fp32(scale):
    """eps counts beside small norms; subnormals and the top of the range are in range."""
    x = gradients((2, 20, 50), "f32", 8, scale=scale / 10)
    out = om.orthogonalize(x, eps=0.0)
    for i in range(2):
        check(f64(x[i]), out[i], [ABC] * 5, eps=0.0)
    out = om.orthogonalize(x)
    check(f64(x[0]), out[0], [ABC] * 5)


def test_small_directions_keep_their_place():
    """Singular values over five decades: the rounds on the Gram matrix keep the small ones."""
    r = np.random.default_rng(3)
    for s, l in ((16, 40), (60, 60), (64, 300), (120, 200)):
        u, _ = np.linalg.qr(r.normal(size=(s, s)))
        v, _ = np.linalg.qr(r.normal(size=(l, s)))
        x = torch.tensor(u @ np.diag(np.logspace(0, -5, s)) @ v.T, dtype=torch.float32, device=dev())
        check(f64(x), om.orthogonalize(x), [ABC] * 5)


def test_zeros_nan_and_infinity_stay_in_their_matrix():
    for s, l in ((16, 60), (64, 100), (100, 140)):
        x = gradients((5, s, l), "f32", s)
        want = om.orthogonalize(x)
        x[1] = 0
        x[2, 3, 7] = float("nan")
        x[3, s - 1, l - 1] = float("inf")
        out = om.orthogonalize(x)
        assert not out[1].any() and out[2].isnan().all() and out[3].isnan().all()
        assert torch.equal(out[0], want[0]) and torch.equal(out[4], want[4])


def test_empty_and_single():
    for shape in ((0, 4, 5), (3, 0, 5), (3, 4, 0), (2, 0, 4, 5)):
        x = torch.empty(shape, device=dev())
        assert om.orthogonalize(x).shape == x.shape
    x = torch.tensor([[[-3.0]]], device=dev())
    check(f64(x[0]), om.orthogonalize(x)[0], [ABC] * 5)


def test_many_matrices():
    """More matrices than a batch of the largest size has, each as it is alone."""
    x = gradients((2300, 70, 72), "bf16", 9)
    out = om.orthogonalize(x)
    for i in (0, 1, 2047, 2048, 2299):
        check(f64(x[i]), out[i], [ABC] * 5)
    x = gradients((3000, 3, 5), "f32", 10)
    out = om.orthogonalize(x)
    for i in (0, 1500, 2999):
        check(f64(x[i]), out[i], [ABC] * 5)


def test_agrees_with_the_bf16_rounds():
    """The other form of the same operator: within its bf16 rounding (3e-2 in relative norm)."""
    x = gradients((2, 128, 768), "f32", 11)
    out = om.orthogonalize(x)
    for i in range(2):
        other = om.zeropower_via_newtonschulz5(x[i], out_dtype=torch.float32)
        assert float((other - out[i]).norm() / out[i].norm()) <= 3e-2


def test_captured_and_replayed():
    x = gradients((7, 100, 300), "bf16", 12)
    om.orthogonalize(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = om.orthogonalize(x)
    for k in range(4):
        x.copy_(gradients((7, 100, 300), "bf16", 20 + k))
        g.replay()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, om.orthogonalize(x)), k


def test_two_streams_at_once():
    x, y = gradients((40, 64, 500), "f32", 13), gradients((9, 128, 200), "f32", 14)
    want = om.orthogonalize(x), om.orthogonalize(y)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        with torch.cuda.stream(s):
            u = om.orthogonalize(x)
        with torch.cuda.stream(t):
            v = om.orthogonalize(y)
        got.append((u, v))
    torch.cuda.synchronize()
    assert all(torch.equal(u, want[0]) and torch.equal(v, want[1]) for u, v in got)


def test_refusals():
    x = gradients((2, 8, 16), "f32", 15)
    for bad in (x[:, :, ::2], x[0, 0], torch.zeros(2, 129, 130, device=dev()), x.cpu()):
        with pytest.raises((ValueError, om.MuonError)):
            om.orthogonalize(bad)
    with pytest.raises(TypeError):
        om.orthogonalize(x.half())
    with pytest.raises(ValueError):
        om.orthogonalize(x.clone().requires_grad_())
    with pytest.raises(ValueError):
        om.orthogonalize(x, out=x[:1])
    with pytest.raises(om.MuonError):
        om.orthogonalize(x, out=x.transpose(0, 1).contiguous().transpose(0, 1)[:, :, :].as_strided(x.shape, (0, 16, 1)))
    with pytest.raises(om.MuonError):
        om.orthogonalize(x[:, :, 1:], out=x[:, :, :-1])
    with pytest.raises(om.MuonError):
        om.orthogonalize(x, steps=-1)
    with pytest.raises(om.MuonError):
        om.orthogonalize(x, eps=float("nan"))
    with pytest.raises(ValueError):
        om.orthogonalize(x, steps=2, schedule=CASCADE)
