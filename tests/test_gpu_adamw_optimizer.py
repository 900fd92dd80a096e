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
