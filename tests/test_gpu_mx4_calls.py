"""GPU tests of how a program may call the linear layer in microscaled 4-bit values and go on with its
results. What it computes is compared bit by bit with the plain call's, which test_gpu_mx4_linear
compares with the oracle.
"""
import pytest
import torch

import orthogonalized_momentum_optimizer_amd as om
from test_gpu_mx4_linear import case, dev, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("shape", [(64,), (6, 64), (2, 3, 64), (2, 1, 3, 64), (0, 3, 64)])
def test_the_result_may_be_changed_in_place(shape, held):
    """y += bias, relu_(y): as after any layer."""
    x = normal(shape, "f32", 1).requires_grad_()
    w, bias = normal((40, 64), "f32", 2).requires_grad_(), normal((40,), "f32", 3).requires_grad_()
    copies = om.MX4Copies([w])[w] if held else None
    dy = normal(shape[:-1] + (40,), "f32", 4)
    want = torch.relu(om.mx4_linear(x, w, copies) * 2 + bias)
    grads = torch.autograd.grad(want, (x, w, bias), dy)
    y = om.mx4_linear(x, w, copies)
    y *= 2
    y += bias
    torch.relu_(y)
    assert torch.equal(y, want)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y, (x, w, bias), dy), grads))
    with torch.no_grad():
        y = om.mx4_linear(x, w, copies)
    y.mul_(2).add_(bias)                          # made without a graph, changed with one
    torch.relu_(y)
    assert torch.equal(y, want)
    assert torch.equal(torch.autograd.grad(y, bias, dy)[0], grads[2])


@pytest.mark.parametrize("shape", [(64,), (6, 64), (2, 3, 64)])
def test_values_and_gradients_made_without_a_graph_may_be_changed_with_one(shape):
    x, b = normal(shape, "f32", 1), normal((40, 64), "f32", 2)
    p = torch.ones((), device=dev(), requires_grad=True)
    with torch.no_grad():
        q = om.mx4_quantize(x)
        values, y = q.dequantize(torch.float32), om.mx4_matmul(q, om.mx4_quantize(b), torch.float32)
    dx, = torch.autograd.grad(om.mx4_linear(x.requires_grad_(), b).sum(), x)
    assert values.shape == x.shape and y.shape == shape[:-1] + (40,) and dx.shape == x.shape
    for t in (values, y, dx):
        want = t + p
        t += p
        assert torch.equal(t, want)
        t.sum().backward()
    assert float(p.grad) == values.numel() + y.numel() + dx.numel()


def test_a_second_derivative_is_refused_also_of_constant_gradients():
    """A penalty on dx depends on the weight though dy does not: refused, not left out of the gradient."""
    x, w, dy = case(8, 64, 40, "f32", "f32")
    y = om.mx4_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy, create_graph=True)
    want = torch.autograd.grad(om.mx4_linear(x, w), (x, w), dy)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    for penalty in (dx.square().sum(), dw.square().sum()):
        with pytest.raises(RuntimeError, match="once"):
            (om.mx4_linear(x, w).sum() + penalty).backward()
    # a function of constants alone: nothing to refuse
    dx, = torch.autograd.grad(om.mx4_linear(x, w.detach()).sum(), x, create_graph=True)
    dw, = torch.autograd.grad(om.mx4_linear(x.detach(), w).sum(), w, create_graph=True)
    assert not dx.requires_grad and not dw.requires_grad


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_operands_may_lie_in_any_way(dtype):
    """Permuted activations, sliced columns, expanded ones, negated views."""
    w = normal((40, 64), dtype, 1)
    base = normal((5, 64, 7), dtype, 2)
    pairs = torch.complex(normal((6, 64), "f32", 3), normal((6, 64), "f32", 4)).conj()
    for x in (base.permute(0, 2, 1), base.permute(2, 0, 1), normal((4, 5, 128), dtype, 5)[:, 1:4, ::2],
              normal((3, 1, 64), dtype, 6).expand(3, 4, 64), normal((64, 9), dtype, 7).t(), normal((), dtype, 8).expand(6, 64),
              *([pairs.imag] if dtype == "f32" else [])):
        v = torch.empty_strided((40, 64), (1, 100), dtype=w.dtype, device=dev()).copy_(w)
        wide = torch.empty((40, 128), dtype=w.dtype, device=dev())[:, ::2].copy_(w)
        dy = normal((40,) + tuple(x.shape[:-1]), dtype, 9).movedim(0, -1)
        flat = x.detach().clone(memory_format=torch.contiguous_format).requires_grad_()
        w.requires_grad_()
        want = om.mx4_linear(flat, w)
        grads = torch.autograd.grad(want, (flat, w), dy.clone(memory_format=torch.contiguous_format))
        x = x.detach().requires_grad_()
        for u in (w, v.requires_grad_(), wide.requires_grad_()):
            y = om.mx4_linear(x, u)
            assert torch.equal(y, want)
            assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(y, (x, u), dy), grads))
        w.requires_grad_(False)


def test_muon_looks_at_its_copies_before_it_steps():
    w = torch.nn.Parameter(normal((96, 64), "bf16", 1))
    for wrong in ([w], w, om.MX4Copies, om.MX4Copies([w])[w], object()):
        with pytest.raises(TypeError):
            om.Muon([w], mx4_copies=wrong)
    other = normal((32, 64), "bf16", 2)
    opt = om.Muon([w], mx4_copies=om.MX4Copies([w, other]))
    w.grad = normal((96, 64), "bf16", 3)
    before = w.detach().clone()
    for bad, error in ((normal((33, 64), "bf16", 4), ValueError), (normal((32, 64), "f32", 4).half(), TypeError)):
        good, other.data = other.data, bad
        with pytest.raises(error):
            opt.step()
        assert torch.equal(w, before) and not opt.state
        other.data = good
    opt.step()
    assert not torch.equal(w, before) and torch.equal(opt.mx4_copies[w][0].data, om.mx4_quantize(w).data)
    om.Muon([w], mx4_copies=om.MX4Copies([])).step()       # nothing held


@pytest.mark.parametrize("held", [False, True])
def test_recomputed_and_offloaded_passes(held):
    """Activations that are recomputed in the backward pass, or wait for it on the host."""
    from torch.utils.checkpoint import checkpoint
    x, w, _ = case(24, 64, 64, "bf16", "bf16")
    copies = om.MX4Copies([w])[w] if held else None

    def net(x):
        return om.mx4_linear(torch.relu(om.mx4_linear(x.view(4, 6, 64), w, copies)), w, copies).float().square().mean()
    want = torch.autograd.grad(net(x), (x, w))
    for reentrant in (False, True):
        x.grad = w.grad = None
        checkpoint(net, x, use_reentrant=reentrant).backward()
        assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])
    with torch.autograd.graph.save_on_cpu():
        got = torch.autograd.grad(net(x), (x, w))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_modes():
    """Inference mode, autocast, forward-mode and functional transforms."""
    x, w, dy = case(24, 64, 40, "bf16", "bf16")
    want = om.mx4_linear(x, w).detach()
    with torch.inference_mode():
        copies = om.MX4Copies([w])
        copies.refresh()
        y = om.mx4_linear(x, w, copies[w])
        z = om.mx4_linear(x.clone(), w)
        h = om.orthogonalize(x.view(2, 12, 64).clone(), steps=20)
    assert torch.equal(y, want) and torch.equal(z, want) and h.isfinite().all()
    copies.refresh()
    with torch.autocast("cuda", torch.bfloat16):
        assert torch.equal(om.mx4_linear(x, w), want)
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        with pytest.raises(RuntimeError):
            om.mx4_linear(forward_ad.make_dual(x.detach(), x.detach()), w)
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda v: om.mx4_linear(x.detach(), v).sum())(w.detach())
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda v: om.mx4_linear(v, w.detach()))(x.detach().view(4, 6, 64))
    with pytest.raises(RuntimeError):
        torch.func.vmap(om.orthogonalize)(x.detach().view(4, 6, 64))
