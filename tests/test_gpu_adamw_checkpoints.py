"""Steps of AdamW from states that torch.optim.AdamW saved, against the float64 oracle."""
import numpy as np
import pytest
import torch

import adamw_ref
import oracle.adamw as oa
import orthogonalized_momentum_optimizer_amd as om
from test_gpu_adamw import E32, f64, on, u8

pytestmark = pytest.mark.gpu
SHAPES = [(300, 17), (5,), (4097,)]


def saved_by_torch(dt, seed):
    """Parameters after three steps of torch.optim.AdamW and its state dict."""
    r = np.random.default_rng(seed)
    ps = [torch.nn.Parameter(on(r.normal(0, 0.5, s), dt)) for s in SHAPES]
    theirs = torch.optim.AdamW(ps, lr=1e-2, betas=(0.9, 0.99), weight_decay=0.1, foreach=False)
    for _ in range(3):
        for p in ps:
            p.grad = on(r.normal(0, 1, p.shape), dt)
        theirs.step()
    return r, ps, theirs.state_dict()


def values(st, n):
    """(m, v) that a state stands for, in float64."""
    if "exp_avg_scale" not in st:
        return f64(st["exp_avg"]), f64(st["exp_avg_sq"])
    m, root = (oa.held(adamw_ref.e4m3_values(adamw_ref.rows(u8(st[k]), np.uint8)),
                       adamw_ref.scale_values(u8(st[k + "_scale"])), n)
               for k in ("exp_avg", "exp_avg_sq"))
    return m, root ** 2


def step_and_compare(opt, ps, r, t):
    """One step; u is at most 10 for these betas and off by at most 40 roundings of it."""
    prev = [(f64(opt.state[p]["master"] if "master" in opt.state[p] else p),
             *values(opt.state[p], p.numel())) for p in ps]
    for p in ps:
        p.grad = on(r.normal(0, 1, p.shape), p.dtype)
    opt.step()
    torch.cuda.synchronize()
    for p, (p0, m0, v0) in zip(ps, prev):
        st = opt.state[p]
        assert st["step"] == t
        f = lambda x: float(np.float32(x))  # noqa: E731
        want = oa.adamw_step(p0, f64(p.grad), m0, v0, t, f(1e-2), f(0.9), f(0.99), f(1e-8), f(0.1))[0]
        got = f64(st["master"]) if "master" in st else f64(p)
        half = 2.0 ** -8 if p.dtype == torch.bfloat16 and "master" not in st else 0.0
        assert np.all(np.abs(got - want) <= (half + 2 * E32) * np.abs(want) + 1e-2 * 400 * E32)
        if "master" in st:
            assert torch.equal(p.detach(), st["master"].to(p.dtype))


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("saved_dt", [torch.bfloat16, torch.float32], ids=str)
def test_steps_from_moments_of_torch_adamw(saved_dt, state_bits):
    """bf16 parameters go on from moments that were saved beside bf16 or fp32 ones."""
    print(f"[adamw] moments of torch, {saved_dt}, {state_bits} bits", flush=True)
    r, ps, saved = saved_by_torch(saved_dt, 21)
    qs = [torch.nn.Parameter(p.detach().to(torch.bfloat16)) for p in ps]
    opt = om.AdamW(qs, state_bits=state_bits)
    saved["param_groups"][0]["state_bits"] = state_bits
    opt.load_state_dict(saved)
    for i, q in enumerate(qs):
        m, v = values(opt.state[q], q.numel())
        m0, v0 = f64(saved["state"][i]["exp_avg"]), f64(saved["state"][i]["exp_avg_sq"])
        if state_bits == 32:
            assert np.array_equal(m, m0) and np.array_equal(v, v0)
        else:
            (y, s), (z, w) = oa.hold(m0), oa.hold(np.sqrt(v0.astype(np.float32)), floor=True)
            assert np.array_equal(m, oa.held(y, s, q.numel()))
            assert np.array_equal(v, oa.held(z, w, q.numel()) ** 2)
    for t in (4, 5):
        step_and_compare(opt, qs, r, t)


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("saved_dt", [torch.bfloat16, torch.float32], ids=str)
def test_masters_beside_states_of_torch_adamw(saved_dt, state_bits):
    print(f"[adamw] masters beside states of torch, {saved_dt}, {state_bits} bits", flush=True)
    r, ps, saved = saved_by_torch(saved_dt, 22)
    qs = [torch.nn.Parameter(p.detach().to(torch.bfloat16)) for p in ps]
    opt = om.AdamW(qs, state_bits=state_bits, master_weights=True)
    saved["param_groups"][0].update(state_bits=state_bits, master_weights=True)
    opt.load_state_dict(saved)
    assert all(torch.equal(opt.state[q]["master"], q.detach().float()) for q in qs)
    for t in (4, 5):
        step_and_compare(opt, qs, r, t)
    assert any(not torch.equal(opt.state[q]["master"], q.detach().float()) for q in qs)
    with torch.no_grad():
        qs[0].fill_(0.25)
    opt.refresh_masters()
    assert bool((opt.state[qs[0]]["master"] == 0.25).all())
