"""Lists longer than one launch, or than one stage of the lookup, takes: AdamW kernels of one
dtype form over up to 1000 tensors (480 a launch, two stages beyond 64), the norm (240 a launch)
and the scaling in place (160), every tensor against the oracle."""
import math

import numpy as np
import pytest
import torch

import oracle.adamw as oa
import orthogonalized_momentum_optimizer_amd as om
from test_gpu_adamw import DT, E32, MODES, Set, dev, f64, norm_bound, on

pytestmark = pytest.mark.gpu


def sizes_of(n, seed):
    """n sizes: most within a block or two of either kernel, some of several, some empty."""
    r = np.random.default_rng(seed)
    sizes = r.integers(1, 700, n)
    sizes[r.random(n) < 0.1] = r.integers(4000, 13000)
    sizes[r.random(n) < 0.05] = 0
    sizes[[0, n - 1]] = 5, 4097
    return [int(x) for x in sizes]


@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
@pytest.mark.parametrize("n,form", [(16, 0), (17, 1), (64, 0), (65, 1), (480, 1), (481, 0), (512, 4), (1000, 1), (1000, 5)])
def test_adamw_over_long_lists(n, form, small):
    """Tensors without elements take no place in a launch, so that the split lies behind 480."""
    pdt, gdt, master = MODES[form]
    print(f"[adamw lists] {n} tensors p={pdt} g={gdt} master={master} small={small}", flush=True)
    sizes = sizes_of(n, n)
    if n in (480, 481):
        sizes = [max(x, 1) for x in sizes]
    s = Set(sizes, pdt, gdt, master, small, seed=n, muls=(1.0, 0.0, 3.0, 0.5, 2.0, 7.0, 0.25))
    r = np.random.default_rng(n + 1)
    for t, scale in ((1, None), (2, 0.37)):
        g = s.grads()
        for i in [int(x) for x in r.integers(0, n, n // 20)] + [k for k in (478, 479, 480, 482) if k < n][t::2]:
            g[i] = None
        cfg = om.make_adamw_config(1e-2, (0.9, 0.99), 1e-8, 0.1, t, seed=t)
        s.step_and_check(cfg, g, None if scale is None else on(scale, torch.float32), f"step {t}")


@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
def test_a_launch_whose_gradients_are_all_absent(small):
    """The first, the middle or the last of three launches has nothing to do."""
    print(f"[adamw lists] absent launches small={small}", flush=True)
    n = 1200
    s = Set([3 + i % 500 for i in range(n)], "bf16", "bf16", False, small, seed=3)
    for t, (lo, hi) in enumerate(((0, 480), (480, 960), (960, 1200), (1, 1199)), 1):
        g = [None if lo <= i < hi else x for i, x in enumerate(s.grads())]
        s.step_and_check(om.make_adamw_config(1e-2, step=t, seed=t), g, label=f"step {t}")


@pytest.mark.parametrize("n", [64, 65, 239, 240, 241, 500, 961])
def test_norm_over_long_lists(n):
    print(f"[norm lists] {n} gradients", flush=True)
    r = np.random.default_rng(n)
    sizes = sizes_of(n, n)
    for k in (n // 2, n - 1):
        sizes[k] = 100001                        # several parts
    gs = [on(r.normal(0, 1, k) * 10.0 ** r.uniform(-6, 2), DT[("f32", "bf16")[i % 2]])
          for i, k in enumerate(sizes)]
    plan = om.GradNormPlan(gs)
    for absent in ((), range(0, n, 7), range(1, n)):
        given = [None if i in absent else g for i, g in enumerate(gs)]
        want, _, each = oa.grad_norm([np.zeros(0) if g is None else f64(g) for g in given])
        for max_norm in (math.inf, want / 3):
            norm, scale, norms = plan.norm(given, max_norm, per_tensor=True)
            assert abs(float(norm) - want) <= norm_bound(want)
            expect = 1.0 if want <= max_norm else max_norm / want
            assert abs(float(scale) - expect) <= 3 * E32 * expect
            assert np.all(np.abs(f64(norms) - each) <= norm_bound(each))
            two = plan.norm(given, max_norm)
            assert torch.equal(two[0], norm) and torch.equal(two[1], scale)


@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [64, 65, 160, 161, 400])
def test_scale_in_place_over_long_lists(n, gdt):
    print(f"[norm lists] scaling {n} gradients {gdt}", flush=True)
    r = np.random.default_rng(n)
    gs = [on(r.normal(0, 1, k), DT[gdt]) for k in sizes_of(n, n)]
    gs += [on(r.normal(0, 1, 9), DT["f32"])]                # and one of another dtype
    was = [g.clone() for g in gs]
    absent = set(range(3, n, 11)) | ({159, 161} & set(range(n)))
    plan = om.GradNormPlan(gs)
    plan.scale_([None if i in absent else g for i, g in enumerate(gs)], on(0.3, torch.float32))
    torch.cuda.synchronize()
    for i, (g, w) in enumerate(zip(gs, was)):
        # one fp32 product, rounded once more in bf16
        want = w if i in absent else (w.float() * torch.tensor(0.3, device=dev())).to(w.dtype)
        assert torch.equal(g, want), i
