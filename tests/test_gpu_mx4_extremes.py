"""GPU tests of the 4-bit operators and of the stacked orthogonalisation at the ends of what they take:
offsets past 32 bits, addresses aligned to an element only, streams, workspaces of two graphs, neighbours
of results, and autograd's view of them. Comparisons are of equal bits: both sides do the same arithmetic."""
import ctypes

import pytest
import torch

import orthogonalized_momentum_optimizer_amd as om
from orthogonalized_momentum_optimizer_amd import _lib as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev():
    return torch.device("cuda", 0)


def noise(*shape, dtype="bf16", seed=0):
    g = torch.Generator(dev()).manual_seed(seed)
    return torch.randn(*shape, device=dev(), generator=g).to(DT[dtype])


def stream():
    return torch.cuda.current_stream().cuda_stream


# ---- offsets past 32 bits ------------------------------------------------------------------------

def test_quantize_and_back_past_32_bits():
    rows, cols = 65552, 65536                               # 8.6 GB; 1025 rows lie past 2^32 elements
    x = torch.zeros(rows, cols, device=dev(), dtype=torch.bfloat16)
    last = noise(32, cols, seed=1)
    x[-32:] = last
    q, t = om.mx4_quantize_both(x)
    want = om.mx4_quantize(last).dequantize()
    back = q.dequantize()
    assert torch.equal(back[-32:], want) and not back[:-32].any()
    del back
    back = t.dequantize()                                   # cols x rows: blocks are of 32 rows of x
    at = rows - rows % 32 - 32                              # (the last rows begin in the middle of one)
    assert torch.equal(back[:, at:], om.mx4_quantize_both(x[at:])[1].dequantize()) and not back[:, :at].any()


def test_product_past_32_bits():
    m, n, k = 65600, 65600, 128                             # 4.3 G results, 8.6 GB
    a, b = noise(m, k, seed=2), noise(n, k, seed=3)
    out = om.mx4_matmul(om.mx4_quantize(a), om.mx4_quantize(b))
    qa = om.mx4_quantize(a[-64:])
    assert torch.equal(out[-64:], om.mx4_matmul(qa, om.mx4_quantize(b)))
    assert torch.equal(out[:64, -128:], om.mx4_matmul(om.mx4_quantize(a[:64]), om.mx4_quantize(b[-128:])))


def test_orthogonalize_past_32_bits():
    far = (1 << 32) + 64                                    # between two matrices, in elements
    store = torch.empty(far + 64 * 100, device=dev(), dtype=torch.bfloat16)
    x = store.as_strided((2, 64, 100), (far, 100, 1))
    values = noise(2, 64, 100, seed=4)
    x.copy_(values)
    want = om.orthogonalize(values)
    om.orthogonalize(x, out=x)
    assert torch.equal(x, want)


# ---- alignment, and what lies next to results ---------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (3, 77, 130), (70, 50, 500), (129, 256, 256), (300, 264, 1000),
                                   (64, 64, 40000)])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_product_into_unaligned_memory(m, n, k, dtype, shift):
    a, b = om.mx4_quantize(noise(m, k, seed=5)), om.mx4_quantize(noise(n, k, seed=6))
    want = om.mx4_matmul(a, b, DT[dtype])
    room = torch.full((m * n + 64 + shift,), 7.0, device=dev(), dtype=DT[dtype])
    out = room[shift + 32:shift + 32 + m * n]
    need = L.muon_mx_matmul_workspace_size(m, n, k)
    ws = torch.full((need + 64,), 255, device=dev(), dtype=torch.uint8)
    codes = [L.muon_mx_codes_size(q.rows, k) for q in (a, b)]
    L.muon_mx_matmul(a.data.data_ptr(), a.data.data_ptr() + codes[0], b.data.data_ptr(),
                     b.data.data_ptr() + codes[1], m, n, k, out.data_ptr(), int(dtype == "f32"), ws.data_ptr(), need,
                     stream())
    assert torch.equal(out.view(m, n), want)
    assert (room[:shift + 32] == 7).all() and (room[shift + 32 + m * n:] == 7).all()
    assert (ws[need:] == 255).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (17, 33), (64, 130), (129, 200)])
@pytest.mark.parametrize("shift", [1, 3])
def test_quantize_and_back_unaligned(rows, cols, dtype, shift):
    store = torch.zeros(rows * (cols + 5) + shift, device=dev(), dtype=DT[dtype])
    x = store[shift:].view(rows, cols + 5)[:, :cols]
    x.copy_(noise(rows, cols, dtype=dtype, seed=7))
    for q, w in zip(om.mx4_quantize_both(x), om.mx4_quantize_both(x.contiguous())):
        assert torch.equal(q.data, w.data)
    q = om.mx4_quantize(x)
    room = torch.full((rows * cols + 64 + shift,), 7.0, device=dev(), dtype=DT[dtype])
    out = room[shift + 32:shift + 32 + rows * cols]
    L.muon_mx_dequantize(q.data.data_ptr(), q.data.data_ptr() + L.muon_mx_codes_size(rows, cols), rows, cols,
                         out.data_ptr(), int(dtype == "f32"), stream())
    assert torch.equal(out.view(rows, cols), q.dequantize(DT[dtype]))
    assert (room[:shift + 32] == 7).all() and (room[shift + 32 + rows * cols:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("count,s,l", [(3, 7, 50), (3, 16, 77), (70, 30, 131), (3, 64, 300), (300, 64, 66),
                                       (2, 100, 1500), (5, 33, 1100), (2, 16, 1500)])
def test_orthogonalize_in_a_larger_tensor(count, s, l, tall, dtype):
    """Rows apart, an odd start, and neighbours that stay as they are; NaN next to the stack is not read."""
    r, c = (l, s) if tall else (s, l)
    values = noise(count, r, c, dtype=dtype, seed=8)
    want = om.orthogonalize(values)
    store = torch.full((count, r + 2, c + 3), float("nan"), device=dev(), dtype=DT[dtype])
    x = store[:, 1:-1, 1:-2]
    x.copy_(values)
    out = torch.full((count, r + 1, c + 5), 7.0, device=dev(), dtype=DT[dtype])
    got = om.orthogonalize(x, out=out[:, :-1, 3:-2])
    assert torch.equal(got, want)
    assert (out[:, -1] == 7).all() and (out[:, :, :3] == 7).all() and (out[:, :, -2:] == 7).all()
    om.orthogonalize(x, out=x)
    assert torch.equal(x, want)
    edge = store.clone()
    edge[:, 1:-1, 1:-2] = float("nan")
    assert edge.isnan().all()


def test_orthogonalize_of_one_matrix_seen_often():
    x = noise(24, 70, seed=9)
    got = om.orthogonalize(x.expand(5, 24, 70))
    one = om.orthogonalize(x)
    assert all(torch.equal(g, one) for g in got)


# ---- streams and graphs -----------------------------------------------------------------------------

def test_calls_follow_the_current_stream():
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=dev())
    a, b = noise(64, 9000, seed=10), noise(64, 9000, seed=11)
    h = noise(2, 128, 1500, seed=12)
    want = om.mx4_matmul(om.mx4_quantize(a), om.mx4_quantize(b)), om.orthogonalize(h)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        late = a.clone()
        late.zero_()
        for _ in range(10):
            big = torch.tanh(big @ big)                     # what the calls have to wait for
        late.copy_(a)
        got = om.mx4_matmul(om.mx4_quantize(late), om.mx4_quantize(b)), om.orthogonalize(h)
    torch.cuda.current_stream().wait_stream(side)
    for w, g in zip(want, got):
        assert torch.equal(w, g)


def test_two_graphs_replayed_at_once():
    """Each graph has its own workspaces: a split product's and a stack's."""
    data = [(noise(64, 40000, seed=20 + i), noise(64, 40000, seed=30 + i), noise(4, 128, 1500, seed=40 + i))
            for i in range(2)]

    def work(a, b, h):
        return om.mx4_matmul(om.mx4_quantize(a), om.mx4_quantize(b), torch.float32), om.orthogonalize(h)
    want = [work(*d) for d in data]
    graphs, outs = [], []
    for d in data:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(work(*d))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(5):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(x, y) for x, y in zip(w, o))


# ---- autograd -------------------------------------------------------------------------------------

def test_out_counts_as_changed():
    w = noise(16, 40, dtype="f32", seed=13)
    x = noise(16, 40, dtype="f32", seed=14).requires_grad_()
    y = (x * w).sum()
    om.orthogonalize(w, out=w)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_linear_refuses_other_devices():
    x, w = noise(8, 32, seed=15), noise(16, 32, seed=16)
    copies = om.MX4Copies([w])
    with pytest.raises(ValueError):
        om.mx4_linear(x, w.cpu(), copies[w])
    with pytest.raises(ValueError):
        om.mx4_linear(x.cpu(), w)


def test_linear_is_differentiable_once():
    x = noise(8, 32, dtype="f32", seed=17).requires_grad_()
    w = noise(16, 32, dtype="f32", seed=18).requires_grad_()
    dx, = torch.autograd.grad(om.mx4_linear(x, w).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        dx.sum().backward()


def test_linear_twice_and_without_tokens_or_outputs():
    x = noise(5, 64, dtype="f32", seed=19).requires_grad_()
    w = noise(48, 64, dtype="f32", seed=20).requires_grad_()
    y = om.mx4_linear(om.mx4_linear(x, w) @ w.detach(), w)  # the same weight twice: gradients add up
    dy = noise(5, 48, dtype="f32", seed=21)
    dx, dw = torch.autograd.grad(y, (x, w), dy, retain_graph=True)
    again = torch.autograd.grad(y, (x, w), dy)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    empty = noise(0, 64, dtype="f32").requires_grad_()
    z = noise(5, 0, dtype="f32").requires_grad_()
    v = noise(48, 0, dtype="f32").requires_grad_()
    gx, gw = torch.autograd.grad(om.mx4_linear(empty, w).sum(), (empty, w))
    assert gx.shape == (0, 64) and gw.shape == (48, 64) and not gw.any()
    y = om.mx4_linear(z, v)
    assert y.shape == (5, 48) and not y.any()
    gz, gv = torch.autograd.grad(y.sum(), (z, v))
    assert gz.shape == (5, 0) and gv.shape == (48, 0)


def test_a_list_of_all_kinds():
    """61 and more sources of both types, wanted as they lie, transposed and both, in one call."""
    xs = [noise(1 + 7 * i % 150, 1 + 13 * i % 200, dtype="bf16" if i % 3 else "f32", seed=i) for i in range(150)]
    entries, kept = [], []
    for i, x in enumerate(xs):
        r, c = x.shape
        bufs = []
        for rows, cols, on in ((r, c, i % 4 != 1), (c, r, i % 4 != 2)):
            n = L.muon_mx_codes_size(rows, cols)
            d = torch.full((n // 16 * 17,), 99, dtype=torch.uint8, device=dev())
            bufs.append(d)
            kept.append((d, on, x if (rows, cols) == (r, c) and len(bufs) == 1 else x.t()))
            bufs.append((d.data_ptr(), d.data_ptr() + n) if on else (None, None))
        entries.append((x.data_ptr(), r, c, c, int(x.dtype == torch.float32), *bufs[1], *bufs[3]))
    a = L.make_mx_sources(entries)
    L.muon_mx_quantize(a, len(entries), 1, ctypes.c_uint64(12345).value, stream())
    for d, on, x in kept:
        if on:
            assert torch.equal(d, om.mx4_quantize(x, stochastic=True, seed=12345).data)
        else:
            assert (d == 99).all()
