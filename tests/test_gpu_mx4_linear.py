"""GPU tests of the linear layer in microscaled 4-bit values: its three products against the float64
oracle and against differences, the held weights that Muon refreshes, graphs, streams and refusals.

Held values are the oracle's, bit by bit, so that only the products' sums and the last rounding
differ: with s the sum of |a b| over k terms, 2 k 2^-24 s for the fp32 sum and 2^-8 of a bf16 result.
"""
import numpy as np
import pytest
import torch

import oracle.mx4 as mx
import orthogonalized_momentum_optimizer_amd as om

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev():
    return torch.device("cuda", 0)


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(shape, dtype, seed, scale=1.0):
    r = np.random.default_rng(seed)
    return torch.tensor(r.normal(0, scale, shape), dtype=torch.float64).to(DT[dtype]).to(dev())


def near(got, a, b):
    """got against a b^T of held values (numpy)."""
    want, s = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = 2 * a.shape[1] * 2.0 ** -24 * s + (2.0 ** -8 * np.abs(want) if got.dtype == torch.bfloat16 else 0)
    err = np.abs(f64(got).reshape(want.shape) - want)
    assert (err <= tol).all(), (err - tol).max()


def case(t, i, o, xd, wd, seed=0):
    x = normal((t, i), xd, seed).requires_grad_()
    w = normal((o, i), wd, seed + 1, 0.02).requires_grad_()
    dy = normal((t, o), xd, seed + 2, 1e-3)
    return x, w, dy


@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("xd,wd", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("t,i,o", [(1, 1, 1), (1, 64, 48), (7, 33, 130), (97, 129, 65), (256, 768, 300),
                                   (1500, 96, 200), (640, 500, 1030)])
def test_three_products_match_the_oracle(t, i, o, xd, wd, stochastic):
    x, w, dy = case(t, i, o, xd, wd)
    y = om.mx4_linear(x, w, stochastic=stochastic, seed=99)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert (y.dtype, dx.dtype, dw.dtype) == (DT[xd], DT[xd], DT[wd])
    seed = 99 if stochastic else None
    X, W, D = f64(x), f64(w), f64(dy)
    near(y, mx.hold(X), mx.hold(W))
    near(dx, mx.hold(D, seed), mx.hold(W.T))
    near(dw, mx.hold(D.T, seed), mx.hold(X.T))


def test_gradients_against_differences():
    """On values that 4 bits hold exactly the layer is bilinear from one grid value to the next: the
    differences of <y, dy> there are the gradients, to the last bit."""
    r = np.random.default_rng(3)
    grid = np.array([-4.0, -2.0, -1.0, -0.5, 0.5, 1.0, 2.0])       # each has a neighbour to go to
    t, i, o = 40, 64, 32
    draw = lambda *s: torch.tensor(r.choice(grid, s), dtype=torch.float32, device=dev())  # noqa: E731
    x, w, dy = draw(t, i), draw(o, i), draw(t, o)
    for m in (x, w, dy):                                           # every block, either way, reaches 6
        m[::32], m[:, ::32] = 6.0, 6.0
    x.requires_grad_(), w.requires_grad_()
    loss = lambda x, w: (om.mx4_linear(x, w) * dy).sum(dtype=torch.float64)  # noqa: E731
    dx, dw = torch.autograd.grad(om.mx4_linear(x, w), (x, w), dy)
    base = loss(x, w)
    for k in range(12):
        a, b, c = int(r.integers(t)), int(r.integers(i)), int(r.integers(o))
        x2, w2 = x.detach().clone(), w.detach().clone()
        x2[a, b] *= 2.0 if abs(x2[a, b]) < 1 else 0.5              # (1/4 is no value of the grid)
        w2[c, b] *= 2.0 if abs(w2[c, b]) < 1 else 0.5
        with torch.no_grad():
            assert float(loss(x2, w) - base) == float(dx[a, b] * (x2[a, b] - x[a, b]))
            assert float(loss(x, w2) - base) == float(dw[c, b] * (w2[c, b] - w[c, b]))


def test_parts_of_the_gradient_and_leading_dimensions():
    x, w, dy = case(60, 64, 40, "bf16", "bf16")
    y = om.mx4_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    z = om.mx4_linear(x.detach(), w)
    assert torch.equal(z, y) and torch.equal(torch.autograd.grad(z, w, dy)[0], dw)
    z = om.mx4_linear(x, w.detach())
    assert torch.equal(torch.autograd.grad(z, x, dy)[0], dx)
    with torch.no_grad():
        assert torch.equal(om.mx4_linear(x, w), y)
    x3 = x.detach().view(3, 20, 64).requires_grad_()
    z = om.mx4_linear(x3, w)
    assert torch.equal(z, y.view(3, 20, 40))
    a, b = torch.autograd.grad(z, (x3, w), dy.view(3, 20, 40))
    assert torch.equal(a, dx.view(3, 20, 64)) and torch.equal(b, dw)
    v = om.mx4_linear(x[5].detach(), w.detach())
    assert v.shape == (40,) and torch.equal(v, y[5])


def test_gradients_that_are_views():
    """An expanded gradient (of a sum), and one that is a transposed view."""
    x, w, _ = case(50, 32, 48, "f32", "f32")
    ones = torch.ones(50, 48, device=dev())
    want = torch.autograd.grad(om.mx4_linear(x, w), (x, w), ones)
    got = torch.autograd.grad(om.mx4_linear(x, w).sum(), (x, w))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dy = normal((48, 50), "f32", 8)
    want = torch.autograd.grad(om.mx4_linear(x, w), (x, w), dy.t().contiguous())
    got = torch.autograd.grad(om.mx4_linear(x, w), (x, w), dy.t())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_tokens():
    x, w, dy = case(0, 32, 48, "f32", "f32")
    y = om.mx4_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert y.shape == (0, 48) and dx.shape == (0, 32) and dw.shape == (48, 32) and not dw.any()


def test_held_weights_follow_refresh():
    ps = [torch.nn.Parameter(normal(s, d, k)) for k, (s, d) in enumerate(
        [((40, 64), "bf16"), ((33, 129), "f32"), ((64, 40), "bf16"), ((1, 5), "f32")])]
    copies = om.MX4Copies(ps)
    for p in ps:
        r, c = om.mx4_quantize_both(p)
        assert torch.equal(copies[p][0].data, r.data) and torch.equal(copies[p][1].data, c.data)
    x, _, dy = case(20, 64, 40, "bf16", "bf16")
    y = om.mx4_linear(x, ps[0], copies[ps[0]])
    z = om.mx4_linear(x, ps[0])
    assert torch.equal(y, z)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y, (x, ps[0]), dy),
                                                 torch.autograd.grad(z, (x, ps[0]), dy)))
    with torch.no_grad():
        ps[0].mul_(3.0)
    old = copies[ps[0]][0].data.clone()
    copies.refresh()
    assert not torch.equal(copies[ps[0]][0].data, old)
    assert torch.equal(copies[ps[0]][0].data, om.mx4_quantize(ps[0]).data)
    ps[0].data = normal((40, 64), "bf16", 77)              # other memory
    copies.refresh()
    assert torch.equal(copies[ps[0]][1].data, om.mx4_quantize(ps[0].t()).data)
    ps[0].data = normal((41, 64), "bf16", 77)
    with pytest.raises(ValueError):
        copies.refresh()


def test_a_backward_pass_over_refreshed_weights_is_refused():
    x, w, dy = case(20, 64, 40, "bf16", "bf16")
    copies = om.MX4Copies([w])
    y = om.mx4_linear(x, w, copies[w])
    copies.refresh()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, (x, w), dy)


def test_many_held_weights_are_one_list():
    """More matrices than one launch takes, of both dtypes."""
    ps = [normal((16 + k % 5, 32 + k), "bf16" if k % 3 else "f32", k) for k in range(150)]
    copies = om.MX4Copies(ps)
    assert len(copies) == 150
    for p in ps:
        r, c = om.mx4_quantize_both(p)
        assert torch.equal(copies[p][0].data, r.data) and torch.equal(copies[p][1].data, c.data)


def test_muon_refreshes_held_weights():
    """Two layers trained as a program would: held weights after each step are the parameters', and
    the parameters those of a Muon that does not know of them."""
    ws = [torch.nn.Parameter(normal((96, 64), "bf16", 1, 0.05)), torch.nn.Parameter(normal((64, 96), "bf16", 2, 0.05))]
    other = [torch.nn.Parameter(w.detach().clone()) for w in ws]
    copies = om.MX4Copies(ws)
    opt, plain = om.Muon(ws, lr=0.05, mx4_copies=copies), om.Muon(other, lr=0.05)
    x = normal((128, 64), "bf16", 3)
    for step in range(3):
        h = torch.relu(om.mx4_linear(x, ws[0], copies[ws[0]], stochastic=True, seed=2 * step))
        om.mx4_linear(h, ws[1], copies[ws[1]], stochastic=True, seed=2 * step + 1).float().square().mean().backward()
        for w, o in zip(ws, other):
            o.grad = w.grad.clone()
        opt.step(), plain.step()
        opt.zero_grad()
        for w, o in zip(ws, other):
            assert torch.equal(w, o)
            r, c = om.mx4_quantize_both(w)
            assert torch.equal(copies[w][0].data, r.data) and torch.equal(copies[w][1].data, c.data)


def test_forward_and_backward_in_a_graph():
    """Captured once, replayed on new inputs with eager work between the replays."""
    x, w, dy = case(300, 128, 96, "bf16", "bf16")
    copies = om.MX4Copies([w])
    step = lambda: torch.autograd.grad(om.mx4_linear(x, w, copies[w], stochastic=True, seed=4), (x, w), dy)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        copies.refresh()
        out = step()
    for k in range(4):
        with torch.no_grad():
            x.copy_(normal((300, 128), "bf16", 50 + k))
            w.copy_(normal((96, 128), "bf16", 60 + k))
            dy.copy_(normal((300, 96), "bf16", 70 + k))
        g.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        want = torch.autograd.grad(om.mx4_linear(x, w, stochastic=True, seed=4), (x, w), dy)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_two_streams_at_once():
    """Split products on two streams have workspaces of their own."""
    a, b = normal((64, 20000), "f32", 1), normal((200, 20000), "f32", 2)
    qa, qb = om.mx4_quantize(a), om.mx4_quantize(b)
    want = om.mx4_matmul(qa, qb, torch.float32), om.mx4_matmul(qb, qa, torch.float32)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s):
            u = om.mx4_matmul(qa, qb, torch.float32)
        with torch.cuda.stream(t):
            v = om.mx4_matmul(qb, qa, torch.float32)
        got.append((u, v))
    torch.cuda.synchronize()
    assert all(torch.equal(u, want[0]) and torch.equal(v, want[1]) for u, v in got)


def test_refusals():
    x, w, dy = case(8, 64, 40, "bf16", "bf16")
    q = om.mx4_quantize(w)
    with pytest.raises(ValueError):
        om.mx4_linear(x[:, :32], w)
    with pytest.raises(TypeError):
        om.mx4_linear(x.half(), w)
    with pytest.raises(TypeError):
        om.mx4_quantize(x.detach().half())
    with pytest.raises(ValueError):
        om.mx4_quantize(x.detach().cpu())
    with pytest.raises(ValueError):
        om.mx4_matmul(q, om.mx4_quantize(x[:, :32].contiguous()))
    with pytest.raises(TypeError):
        om.mx4_matmul(q, w)
    with pytest.raises(TypeError):
        om.mx4_matmul(q, q, torch.float16)
    with pytest.raises(ValueError):
        om.mx4_linear(x, w, (q, q))
    with pytest.raises(ValueError):
        om.MX4Copies([w, w])
    with pytest.raises(ValueError):
        om.MX4Copies([w.t()])
    bad = om.mx4_quantize(w)
    bad.data = bad.data[:-64]
    with pytest.raises(ValueError):
        om.mx4_matmul(bad, bad)
    with pytest.raises(ValueError):
        bad.dequantize()
