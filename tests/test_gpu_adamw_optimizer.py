"""The AdamW optimizer where its groups, gradients or states differ from step to step."""
import numpy as np
import pytest
import torch

import orthogonalized_momentum_optimizer_amd as om
from test_gpu_adamw import on

pytestmark = pytest.mark.gpu


def snapshot(opt):
    return [(p.detach().clone(), {k: v.clone() if torch.is_tensor(v) else v
                                  for k, v in opt.state[p].items()})
            for g in opt.param_groups for p in g["params"]]


def unchanged(opt, was):
    return all(torch.equal(p.detach(), w) and opt.state[p].keys() == st.keys() and
               all(torch.equal(v.view(torch.uint8), st[k].view(torch.uint8)) if torch.is_tensor(v)
                   else v == st[k] for k, v in opt.state[p].items())
               for p, (w, st) in zip([p for g in opt.param_groups for p in g["params"]], was))


@pytest.mark.parametrize("state_bits", [32, 8])
def test_a_refused_step_changes_no_group(state_bits):
    """What the last of the step's calls would refuse (a gradient that starts at 4 bytes or lies in
    a parameter, an option) is found before the first is made; the step can then be taken again."""
    print(f"[adamw] refused in a later group, {state_bits} bits", flush=True)
    r = np.random.default_rng(31)
    sizes = (700, 5000, 301)
    x = [on(r.normal(0, 1, n), torch.float32) for n in sizes]
    g = [on(r.normal(0, 1, n), torch.float32) for n in sizes]
    runs = []
    for refused in (True, False):
        ps = [torch.nn.Parameter(t.clone()) for t in x]
        opt = om.AdamW([{"params": ps[:1]}, {"params": ps[1:]}], lr=1e-2, state_bits=state_bits,
                       weight_decay=0.1)
        for p, t in zip(ps, g):
            p.grad = t.clone()
        ps[2].grad = None
        opt.step()                                    # the last parameter is a step behind
        ps[2].grad = g[2].clone()
        if refused:
            opt.step()
            was = snapshot(opt)
            for bad in (torch.cat([g[2][:1], g[2]])[1:], ps[1].detach()[:301]):
                ps[2].grad = bad
                with pytest.raises(om.MuonError):
                    opt.step()
                torch.cuda.synchronize()
                assert unchanged(opt, was)
            ps[2].grad = g[2].clone()
            opt.param_groups[1]["betas"] = (0.9, 1.0)
            with pytest.raises(om.MuonError):
                opt.step()
            torch.cuda.synchronize()
            assert unchanged(opt, was)
            opt.param_groups[1]["betas"] = (0.9, 0.999)
        else:
            opt.step()
        opt.step()
        torch.cuda.synchronize()
        assert [opt.state[p]["step"] for p in ps] == [3, 3, 2]
        runs.append(snapshot(opt))
    assert all(torch.equal(a, b) for (a, _), (b, _) in zip(*runs))


class Alternating:
    """An optimizer whose steps see a changing set of gradients, beside one optimizer for each
    parameter that steps only where there is one: the same bits after every step."""

    def __init__(self, state_bits, sizes=(700, 5000, 301, 4097)):
        self.r = np.random.default_rng(32)
        dts = [torch.bfloat16, torch.float32] * 2
        self.ps, self.qs = ([torch.nn.Parameter(on(np.random.default_rng(n).normal(0, 1, n), dt))
                             for n, dt in zip(sizes, dts)] for _ in "pq")
        more = dict(lr=1e-2, state_bits=state_bits, weight_decay=0.1, master_weights=True, seed=5)
        self.opt = om.AdamW(self.ps, **more)
        self.alone = [om.AdamW([q], **more) for q in self.qs]

    def gradients(self, live):
        for i, (p, q) in enumerate(zip(self.ps, self.qs)):
            p.grad = q.grad = None
            if i in live:
                p.grad = on(self.r.normal(0, 1, p.numel()), torch.float32).to(q.dtype)
                q.grad = p.grad.clone()

    def plan(self):
        return self.opt._plans[0][0]

    def step(self, live):
        self.gradients(live)
        self.opt.step()
        for opt in self.alone:
            opt.step()
        self.compare()

    def compare(self):
        torch.cuda.synchronize()
        for p, q, opt in zip(self.ps, self.qs, self.alone):
            assert torch.equal(p.detach(), q.detach())
            st, want = self.opt.state.get(p, {}), opt.state.get(q, {})
            assert st.keys() == want.keys()
            for k, v in st.items():
                assert (torch.equal(v.view(torch.uint8), want[k].view(torch.uint8))
                        if torch.is_tensor(v) else v == want[k]), k


@pytest.mark.parametrize("state_bits", [32, 8])
def test_gradients_that_come_and_go_keep_the_plan(state_bits):
    """A new plan for each parameter met for the first time, and none after that."""
    print(f"[adamw] alternating gradients, {state_bits} bits", flush=True)
    a = Alternating(state_bits)
    for live in ([0], [1], [0, 1], [2, 3], [1]):
        a.step(live)
    plan = a.plan()
    assert len(a.opt._plans[0][1]) == 4
    for live in ([0, 1, 2, 3], [3], [0, 2], [1], [], [0, 1, 2, 3], [2, 1]):
        a.step(live)
        assert a.plan() is plan


@pytest.mark.parametrize("state_bits", [32, 8])
def test_absent_parameters_that_move_leave_the_plan(state_bits):
    """...and come back with their next gradient, from where they are then. One that is on the host
    meanwhile does not hinder the others."""
    print(f"[adamw] absent and moved, {state_bits} bits", flush=True)
    a = Alternating(state_bits)
    a.step([0, 1, 2, 3])
    a.ps[1].grad = None
    a.ps[1].data = a.ps[1].data.cpu()
    st = a.opt.state[a.ps[2]]
    for k, v in st.items():
        if torch.is_tensor(v):
            st[k] = v.cpu()
    for _ in range(2):
        a.gradients([0, 3])
        a.opt.step()
        for opt in a.alone:
            opt.step()
    plan = a.plan()
    assert len(a.opt._plans[0][1]) == 2
    a.ps[1].data = a.ps[1].data.cuda()
    for k, v in st.items():
        if torch.is_tensor(v):
            st[k] = v.cuda()
    a.compare()
    a.step([1, 2])
    assert a.plan() is not plan and len(a.opt._plans[0][1]) == 4
    with torch.no_grad():
        a.ps[0].data = a.ps[0].detach().clone()              # another address, no gradient
    a.step([3])
    a.step([0, 1, 2, 3])


@pytest.mark.parametrize("state_bits", [32, 8])
def test_a_step_of_some_gradients_can_be_captured(state_bits):
    """Every parameter has had a step: no state or table is missing. Two graphs of different sets
    in turn, replayed between eager steps of all, each replay against the step that it captured."""
    print(f"[adamw] captured sets, {state_bits} bits", flush=True)
    a = Alternating(state_bits)
    a.step([0, 1, 2, 3])
    a.step([0, 1, 2, 3])
    graphs, held = [], []
    for live in ([0, 2], [1]):
        a.gradients(live)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a.opt.step()
        graphs.append((graph, live))
        held.append([(p.grad, q.grad) for p, q in zip(a.ps, a.qs)])
        for i in live:                               # the replay's index is the captured one
            a.opt.state[a.ps[i]]["step"] -= 1
    for k in range(6):
        graph, live = graphs[k % 2]
        steps = [opt.state[q]["step"] for opt, q in zip(a.alone, a.qs)]
        graph.replay()
        for opt, q, (_, g) in zip(a.alone, a.qs, held[k % 2]):
            q.grad = g
            opt.state[q]["step"] = 2                 # as captured
            opt.step()
        for opt, q, st, n in zip(a.alone, a.qs, [a.opt.state[p] for p in a.ps], steps):
            opt.state[q]["step"] = st["step"] = n
        a.compare()
        if k % 3 == 2:
            a.step([0, 1, 2, 3])


@pytest.mark.parametrize("state_bits", [32, 8])
def test_a_parameter_set_into_an_absent_one_steps(state_bits):
    """The absent one is left out of the plan: no buffer of it stands in the way."""
    print(f"[adamw] live one in an absent one's memory, {state_bits} bits", flush=True)
    a = Alternating(state_bits, sizes=(700, 5000, 700))     # (0 and 2 are bf16)
    a.step([0, 1, 2])
    for ps in (a.ps, a.qs):
        ps[2].data = ps[0].data
    a.step([1, 2])
    assert len(a.opt._plans[0][1]) == 2
    plan = a.plan()
    a.step([2])
    assert a.plan() is plan
    for ps in (a.ps, a.qs):
        ps[2].data = ps[0].detach().clone()
    a.step([0, 1, 2])
    assert len(a.opt._plans[0][1]) == 3
