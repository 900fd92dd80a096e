"""GPU parity of the AdamW step (fp32 and 8-bit states) and of the gradient norm with the
float64 oracle, through the Python front end.

Every step is compared from the stored state before it. fp32 states, with E = 2^-24 (half a
unit in the last place), in units of the magnitudes that are added:
* m: the gradient's scaling, (1 - b1), its product and the final sum round: 4 E;
* v: squaring the scaled gradient doubles its rounding, then the square, (1 - b2), its product
  and the sum: 6 E;
* u = (m / bc1) / (sqrt(v) / sqrt(bc2) + eps): m's error carried over, and 3 E from v under the
  root, the root, two correction factors and their products, the sum with eps, the division,
  the last product: 10 E, taken as 16 E;
* p: 2 E of p (the product with lr and the sum), lr times the errors of u and of the decay, and
  half a bf16 unit (2^-9 of the value's binade, at most 2^-8 p) for a stored bf16 parameter.
A result under 2^-126 is rounded to a multiple of 2^-149 instead, off by at most 2^-150: three
such roundings enter m and v (the square or scaled gradient, the product with 1 - b, the sum;
their factors are at most 1). In v they change sqrt(v) by a factor between sqrt(1 - x) and
sqrt(1 + x), x = 3 2^-150 / v, hence u by at most 1 / sqrt(1 - x) - 1 of itself.
8-bit states are compared byte by byte with the operation-by-operation fp32 evaluation
(adamw_ref.py), which the CPU tests hold to the float64 definition.
"""
import copy
import math

import numpy as np
import pytest
import torch

import adamw_ref
import oracle.adamw as oa
import orthogonalized_momentum_optimizer_amd as om
from orthogonalized_momentum_optimizer_amd import _lib as L

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24
SUB = 3 * 2.0 ** -150
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [0, 1, 7, 8, 15, 16, 17, 255, 256, 257, 511, 4095, 4096, 4097, 8192, 8193, 70001]
MODES = [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "f32", False),
         ("f32", "bf16", False), ("bf16", "bf16", True), ("bf16", "f32", True)]


def dev():
    return torch.device("cuda", 0)


def f64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def u8(t):
    return t.view(torch.uint8).cpu().numpy().reshape(-1)


def on(x, dt):
    return torch.tensor(np.asarray(x), dtype=dt, device=dev())


def zeros8(n, dt):
    return torch.zeros(n, dtype=torch.uint8, device=dev()).view(dt)


class Set:
    """Tensors of the given sizes with their states, and a plan of them."""

    def __init__(self, sizes, pdt, gdt, master, small, seed=0, std=0.5, muls=(1.0, 0.0, 3.0)):
        r = np.random.default_rng(seed)
        self.r, self.sizes, self.small, self.pdt, self.gdt = r, list(sizes), small, pdt, gdt
        self.muls = [muls[i % len(muls)] for i in range(len(self.sizes))]
        self.w = [on(r.normal(0, std, n), torch.float32) for n in sizes] if master else None
        self.p = ([w.to(DT[pdt]) for w in self.w] if master else
                  [on(r.normal(0, std, n), DT[pdt]) for n in sizes])
        more = {}
        if small:
            self.m = [zeros8(n, torch.float8_e4m3fn) for n in sizes]
            self.v = [zeros8(n, torch.float8_e4m3fn) for n in sizes]
            self.ms = [zeros8(-(-n // 256), torch.float8_e8m0fnu) for n in sizes]
            self.vs = [zeros8(-(-n // 256), torch.float8_e8m0fnu) for n in sizes]
            more = dict(exp_avg_scales=self.ms, exp_avg_sq_scales=self.vs)
        else:
            self.m = [torch.zeros(n, device=dev()) for n in sizes]
            self.v = [torch.zeros(n, device=dev()) for n in sizes]
        self.plan = om.AdamWPlan(self.p, self.m, self.v, [DT[gdt]] * len(self.sizes),
                                 masters=self.w, wd_muls=self.muls, **more)

    def grads(self, std=1.0):
        return [on(self.r.normal(0, std, n) * 10.0 ** self.r.uniform(-3, 0, n), DT[self.gdt])
                for n in self.sizes]

    def all(self):
        out = self.p + self.m + self.v + (self.w or [])
        return out + (self.ms + self.vs if self.small else [])

    def bytes(self):
        return [u8(t.contiguous().view(torch.uint8) if t.numel() else
                   torch.zeros(0, dtype=torch.uint8)) for t in self.all()]

    def before(self, i):
        src = self.w[i] if self.w else self.p[i]
        if self.small:
            return (f64(src), u8(self.m[i]), u8(self.ms[i]), u8(self.v[i]), u8(self.vs[i]))
        return f64(src), f64(self.m[i]), f64(self.v[i])

    def check(self, i, prev, g, cfg, scale=1.0, label=""):
        n = self.sizes[i]
        if n == 0:
            return
        g = f64(g)
        if self.small:
            p0, mc, ms, rc, rs = prev
            m0 = oa.held(adamw_ref.e4m3_values(adamw_ref.rows(mc, np.uint8)), adamw_ref.scale_values(ms), n)
            v0 = oa.held(adamw_ref.e4m3_values(adamw_ref.rows(rc, np.uint8)), adamw_ref.scale_values(rs), n) ** 2
            want = adamw_ref.step_codes(g.astype(np.float32), mc, ms, rc, rs, cfg.beta1, cfg.beta2,
                                        cfg.seed, cfg.step, cfg.stochastic, np.float32(scale))
            got = (u8(self.m[i]), u8(self.ms[i]), u8(self.v[i]), u8(self.vs[i]))
            for name, a, b in zip(("m", "m scale", "r", "r scale"), got, want):
                bad = np.flatnonzero(a != b)
                assert bad.size == 0, (f"{label}: {bad.size} bytes of {name} differ, first at "
                                       f"{bad[0]}: {a[bad[0]]} for {b[bad[0]]}")
        else:
            p0, m0, v0 = prev
        lam = cfg.weight_decay * self.muls[i]
        with np.errstate(divide="ignore", invalid="ignore"):
            p, m, v = oa.adamw_step(p0, g, m0, v0, cfg.step, cfg.lr, cfg.beta1, cfg.beta2, cfg.eps,
                                    lam, scale)
        b1, b2, t = cfg.beta1, cfg.beta2, cfg.step
        mag_m = b1 * np.abs(m0) + (1 - b1) * np.abs(scale * g)
        mag_v = b2 * v0 + (1 - b2) * (scale * g) ** 2
        if not self.small:
            assert np.all(np.abs(f64(self.m[i]) - m) <= 4 * E32 * mag_m + SUB), f"{label}: m"
            assert np.all(np.abs(f64(self.v[i]) - v) <= 6 * E32 * mag_v + SUB), f"{label}: v"
        den = np.sqrt(v / (1 - b2 ** t)) + cfg.eps
        with np.errstate(divide="ignore", invalid="ignore"):
            bound_u = np.abs(m) / (1 - b1 ** t) / den
            low = 1 / np.sqrt(np.maximum(1 - SUB / v, 0)) - 1          # infinite: nothing known
            low = np.where(v > 0, low, 0)
            du = np.where(den > 0, (4 * E32 * mag_m + SUB) / (1 - b1 ** t) / den
                          + (16 * E32 + low) * bound_u, 0)
            tol = 2 * E32 * np.abs(p) + cfg.lr * (du + 4 * E32 * abs(lam) * np.abs(p0)) + 1e-30
        if self.w:
            assert np.all(np.abs(f64(self.w[i]) - p) <= tol), f"{label}: master"
            assert torch.equal(self.p[i], self.w[i].to(DT[self.pdt])), f"{label}: p of master"
        else:
            if self.pdt == "bf16":
                tol = tol + 2.0 ** -8 * np.abs(p)
            # (a parameter that an underflowed v and eps = 0 made infinite stays so, or NaN)
            lost = ~np.isfinite(p0) & ~np.isfinite(f64(self.p[i]))
            bad = np.flatnonzero(~(np.abs(f64(self.p[i]) - p) <= tol) & ~lost)
            assert bad.size == 0, f"{label}: {bad.size} parameters, first at {bad[0]}"

    def step_and_check(self, cfg, grads, scale=None, label=""):
        prev = [self.before(i) for i in range(len(self.sizes))]
        self.plan.step(grads, cfg, grad_scale=scale)
        torch.cuda.synchronize()
        s = 1.0 if scale is None else float(scale)
        for i, g in enumerate(grads):
            if g is None:
                now = self.before(i)
                assert all(np.array_equal(a, b) for a, b in zip(prev[i], now))
            else:
                self.check(i, prev[i], g, cfg, s, f"{label} tensor {i} ({self.sizes[i]})")


@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
@pytest.mark.parametrize("pdt,gdt,master", MODES)
def test_steps_over_edge_sizes(pdt, gdt, master, small):
    """Sizes around the vectors, rows, blocks and chunks, three steps with a scale in between."""
    print(f"[adamw] edge sizes p={pdt} g={gdt} master={master} small={small}", flush=True)
    s = Set(SIZES, pdt, gdt, master, small)
    for t, scale, stochastic in ((1, None, True), (2, 0.37, True), (3, None, False)):
        cfg = om.make_adamw_config(1e-2, (0.9, 0.99), 1e-8, 0.1, t, stochastic=stochastic, seed=t)
        s.step_and_check(cfg, s.grads(), None if scale is None else on(scale, torch.float32),
                         f"step {t}")


@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
def test_more_tensors_than_one_launch_mixed_dtypes(small):
    """130 tensors of four dtype pairs with and without masters in one plan; some gradients None."""
    print(f"[adamw] 130 tensors small={small}", flush=True)
    sets = [Set([(i * 977) % 5000 + 1 for i in range(k, 130, 4)], *MODES[k], small, seed=k)
            for k in (0, 1, 3, 4)]
    held = lambda name: [x for s in sets for x in (getattr(s, name) or [None] * len(s.p))]  # noqa: E731
    more = dict(exp_avg_scales=held("ms"), exp_avg_sq_scales=held("vs")) if small else {}
    plan = om.AdamWPlan(held("p"), held("m"), held("v"),
                        [DT[s.gdt] for s in sets for _ in s.p], masters=held("w"),
                        wd_muls=[x for s in sets for x in s.muls], **more)
    cfg = om.make_adamw_config(1e-2, (0.8, 0.95), 1e-10, 0.02, 7, seed=3)
    grads = [s.grads() for s in sets]
    for g in grads:
        g[3] = None
    prev = [[s.before(i) for i in range(len(s.p))] for s in sets]
    plan.step([x for g in grads for x in g], cfg)
    torch.cuda.synchronize()
    for s, g, b in zip(sets, grads, prev):
        for i in range(len(s.p)):
            if g[i] is None:
                assert all(np.array_equal(x, y) for x, y in zip(b[i], s.before(i)))
            else:
                s.check(i, b[i], g[i], cfg, label=f"{s.pdt},{s.gdt} tensor {i}")


@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
def test_rows_behind_the_end_stay(small):
    """Tensors that are views of larger buffers: what follows their last element is not written."""
    print(f"[adamw] behind the end small={small}", flush=True)
    n, room = 4096 + 273, 4096 + 512
    fill = lambda dt: torch.full((room * dt.itemsize,), 0x55, dtype=torch.uint8, device=dev()).view(dt)  # noqa: E731
    p, w = fill(torch.bfloat16), fill(torch.float32)
    mdt = torch.float8_e4m3fn if small else torch.float32
    m, v, ms, vs = fill(mdt), fill(mdt), fill(torch.float8_e8m0fnu), fill(torch.float8_e8m0fnu)
    b = -(-n // 256)
    for x, k in ((p, n), (w, n), (m, n), (v, n), (ms, b), (vs, b)):
        x.view(torch.uint8)[:k * x.element_size()] = 0
    more = dict(exp_avg_scales=[ms[:b]], exp_avg_sq_scales=[vs[:b]]) if small else {}
    plan = om.AdamWPlan([p[:n]], [m[:n]], [v[:n]], [torch.float32], masters=[w[:n]], **more)
    plan.step([torch.randn(n, device=dev())], om.make_adamw_config(step=1))
    torch.cuda.synchronize()
    for x, k in ((p, n), (w, n), (m, n), (v, n)) + (((ms, b), (vs, b)) if small else ()):
        raw = x.view(torch.uint8)
        assert bool((raw[k * x.element_size():] == 0x55).all())
        assert bool(raw[:k * x.element_size()].any())


@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
def test_special_values(small):
    print(f"[adamw] special values small={small}", flush=True)
    n = 5000
    s = Set([n], "f32", "f32", False, small, muls=(0.0,))
    before = s.bytes()
    zero = [torch.zeros(n, device=dev())]
    s.plan.step(zero, om.make_adamw_config(0.1, eps=1e-8, step=1))        # nothing moves
    assert all(np.array_equal(a, b) for a, b in zip(before, s.bytes()))
    for std in (1e-18, 1e-12, 1e-3, 1e6, 1e15):                           # gradients far from 1
        s = Set([n], "f32", "f32", False, small, seed=3)
        for t in (1, 2):
            s.step_and_check(om.make_adamw_config(1e-2, (0.9, 0.99), 0.0, 0.0, t, seed=1),
                             s.grads(std), label=f"std {std} step {t}")
    for std in (1e-30, 1e-36, 1e-41):              # v is zero, m and its scale at the bottom of fp32
        s = Set([n], "f32", "f32", False, small, seed=3)
        for t in (1, 2):
            s.step_and_check(om.make_adamw_config(1e-2, (0.9, 0.99), 1e-8, 0.0, t, seed=1),
                             s.grads(std), label=f"std {std} step {t}")
    s = Set([n], "f32", "f32", False, small, seed=4)                      # a late step
    s.step_and_check(om.make_adamw_config(1e-2, step=10 ** 9, seed=2 ** 63), s.grads())
    s = Set([n], "f32", "f32", False, small, seed=5)                      # no averaging at all
    s.step_and_check(om.make_adamw_config(1e-2, (0.0, 0.0), step=2), s.grads())


@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
def test_nan_and_infinity_stay_in_their_tensor(small):
    print(f"[adamw] nan and infinity small={small}", flush=True)
    sizes = [3000, 3000, 3000]
    s = Set(sizes, "f32", "f32", False, small, seed=6)
    grads = s.grads()
    grads[0][5], grads[0][700] = math.nan, -math.inf
    grads[1][2999] = 1e30                                                 # v overflows, m does not
    for t in (1, 2):
        prev = s.before(2)
        s.plan.step(grads, om.make_adamw_config(step=t, seed=t))
        torch.cuda.synchronize()
        s.check(2, prev, grads[2], om.make_adamw_config(step=t, seed=t))
        bad = torch.isnan(s.p[0])
        assert bool(bad[5]) and bool(bad[700])
        assert bool(torch.isnan(s.m[0].float())[5]) and not bool(torch.isfinite(s.m[0].float())[700])
        ok = torch.ones(3000, dtype=torch.bool, device=dev())
        ok[[5, 700]] = False
        assert not bool(bad[ok].any())                                    # its block loses state only
        assert bool(torch.isfinite(s.p[1]).all())
        held = s.v[1].float() * (torch.repeat_interleave(s.vs[1].float(), 256)[:3000] if small else 1)
        assert float(held[2999]) > (1e17 if small else 1e38)
        if small:
            assert not bool(torch.isnan(s.v[1].float()).any())


@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
def test_skip_of_a_scale_that_is_not_finite(small):
    print(f"[adamw] skip small={small}", flush=True)
    s = Set([1, 4097, 300], "bf16", "bf16", True, small)
    before = s.bytes()
    for bad in (math.nan, math.inf, -math.inf):
        s.plan.step(s.grads(), om.make_adamw_config(step=1, skip_nonfinite=True),
                    grad_scale=on(bad, torch.float32))
        assert all(np.array_equal(a, b) for a, b in zip(before, s.bytes()))
    scale = on(0.5, torch.float32)
    s.step_and_check(om.make_adamw_config(step=1, skip_nonfinite=True), s.grads(), scale)
    s.plan.step(s.grads(), om.make_adamw_config(step=2), grad_scale=on(math.nan, torch.float32))
    assert bool(torch.isnan(s.w[1]).all())                                # without the guard


@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
def test_deterministic_and_independent_of_the_list(small):
    """The same bits twice, and the same for a tensor alone as among others."""
    print(f"[adamw] determinism small={small}", flush=True)
    outs = []
    for order in ([0, 1, 2], [0, 1, 2], [2, 0, 1]):
        s = Set([513, 9001, 12288], "bf16", "bf16", False, small, seed=9)
        g = s.grads()
        more = (dict(exp_avg_scales=[s.ms[i] for i in order], exp_avg_sq_scales=[s.vs[i] for i in order])
                if small else {})
        plan = om.AdamWPlan([s.p[i] for i in order], [s.m[i] for i in order], [s.v[i] for i in order],
                            [torch.bfloat16] * 3, **more)
        for t in (1, 2):
            plan.step([g[i] for i in order], om.make_adamw_config(step=t, seed=4))
        outs.append(s.bytes())
    for other in outs[1:]:
        assert all(np.array_equal(a, b) for a, b in zip(outs[0], other))


def test_offsets_beyond_32_bits():
    """One bf16 tensor of 2^33 + 5000 elements with 8-bit states (50 GB): elements around 2^31,
    2^32, 2^33 and the ends step as they would alone, and the norm counts all of them."""
    n = 2 ** 33 + 5000
    print(f"[adamw] {n} elements", flush=True)
    p, g = (torch.zeros(n, dtype=torch.bfloat16, device=dev()) for _ in "pg")
    m, v = (zeros8(n, torch.float8_e4m3fn) for _ in "mv")
    ms, vs = (zeros8(-(-n // 256), torch.float8_e8m0fnu) for _ in "mv")
    plan = om.AdamWPlan([p], [m], [v], [torch.bfloat16], exp_avg_scales=[ms], exp_avg_sq_scales=[vs])
    cfg = om.make_adamw_config(1e-2, (0.9, 0.99), 1e-8, 0.0, 3, seed=5)
    spans = [(a - 512, a + 512) for a in (2 ** 31, 2 ** 32, 2 ** 33)] + [(0, 1024), (n - 1160, n)]
    r = np.random.default_rng(0)
    for a, b in spans:
        g[a:b] = on(r.normal(0, 1, b - a), torch.bfloat16)
    norm, scale = om.grad_norm([g])
    plan.step([g], cfg)
    torch.cuda.synchronize()
    total = 0.0
    for a, b in spans:
        k, gs = b - a, g[a:b].float().cpu().numpy()
        zc, zs = np.zeros(k, np.uint8), np.zeros(-(-k // 256), np.uint8)
        bits = oa.rounding_bits
        oa.rounding_bits = lambda i, seed, step: bits(np.asarray(i) + a, seed, step)
        try:
            want = adamw_ref.step_codes(gs, zc, zs, zc, zs, cfg.beta1, cfg.beta2, 5, 3, True)
        finally:
            oa.rounding_bits = bits
        got = (u8(m[a:b]), u8(ms[a // 256:-(-b // 256)]), u8(v[a:b]), u8(vs[a // 256:-(-b // 256)]))
        for x, y in zip(got, want):
            assert np.array_equal(x, y), (a, b)
        assert bool((p[a:b] != 0).any())
        total += np.sum(gs.astype(np.float64) ** 2)
    assert int((p != 0).sum()) <= sum(b - a for a, b in spans)            # nothing else moved
    assert abs(float(norm) - math.sqrt(total)) <= 2 * E32 * math.sqrt(total) and float(scale) == 1.0
    del p, g, m, v, plan
    torch.cuda.empty_cache()


def test_fp32_states_of_more_than_one_piece():
    """One bf16 tensor of 2^32 + 5000 elements with fp32 states (51 GB), cut into three pieces:
    elements around the cuts at 2^31 and 2^32 and the ends step as the formula says, no other moves."""
    n = 2 ** 32 + 5000
    print(f"[adamw] {n} elements, fp32 states", flush=True)
    p, g = (torch.zeros(n, dtype=torch.bfloat16, device=dev()) for _ in "pg")
    m, v = (torch.zeros(n, device=dev()) for _ in "mv")
    plan = om.AdamWPlan([p], [m], [v], [torch.bfloat16])
    cfg = om.make_adamw_config(1e-2, (0.9, 0.99), 1e-8, 0.0, 3)
    spans = [(a - 600, a + 600) for a in (2 ** 31, 2 ** 32)] + [(0, 1000), (n - 1160, n)]
    r = np.random.default_rng(1)
    for a, b in spans:
        g[a:b] = on(r.normal(0, 1, b - a), torch.bfloat16)
    plan.step([g], cfg)
    torch.cuda.synchronize()
    for a, b in spans:
        gs = f64(g[a:b])
        want, wm, wv = oa.adamw_step(np.zeros(b - a), gs, np.zeros(b - a), np.zeros(b - a), 3,
                                     cfg.lr, cfg.beta1, cfg.beta2, cfg.eps)
        assert np.all(np.abs(f64(m[a:b]) - wm) <= 4 * E32 * np.abs(wm))
        assert np.all(np.abs(f64(v[a:b]) - wv) <= 6 * E32 * wv)
        assert np.all(np.abs(f64(p[a:b]) - want) <= (2.0 ** -8 + 20 * E32) * np.abs(want))
    total = sum(b - a for a, b in spans)
    assert total - 20 <= int((p != 0).sum()) <= total
    assert int((m != 0).sum()) <= total
    del p, g, m, v, plan
    torch.cuda.empty_cache()


# ---- gradient norm ---------------------------------------------------------------------------

def norm_bound(x):
    """The double sum of n squares is off by at most n 2^-53 of itself (n < 2^22 here), the root
    halves that, and fp32 rounds once."""
    return (E32 + 2.0 ** -31) * abs(x)


@pytest.mark.parametrize("dts", [("f32",), ("bf16",), ("bf16", "f32")])
def test_grad_norm_sizes(dts):
    print(f"[norm] sizes {dts}", flush=True)
    r = np.random.default_rng(1)
    for sizes in (SIZES + [16383, 16384, 16385, 300001], [0], [0, 0, 5], [1], [3] * 150):
        gs = [on(r.normal(0, 1, n) * 10.0 ** r.uniform(-8, 3), DT[dts[i % len(dts)]])
              for i, n in enumerate(sizes)]
        plan = om.GradNormPlan(gs)
        want, _, each = oa.grad_norm(gs)
        for max_norm in (math.inf, want * 2, want / 3, 0.0):
            norm, scale, norms = plan.norm(gs, max_norm, per_tensor=True)
            assert abs(float(norm) - want) <= norm_bound(want)
            expect = 1.0 if want <= max_norm else max_norm / want
            assert abs(float(scale) - expect) <= 3 * E32 * expect
            assert np.all(np.abs(f64(norms) - each) <= norm_bound(each))
            two = plan.norm(gs, max_norm)
            assert torch.equal(two[0], norm) and torch.equal(two[1], scale)
    for empty in ([], [torch.zeros(0, device=dev())]):
        norm, scale, norms = om.GradNormPlan(empty).norm(empty, 1.0, per_tensor=True)
        assert float(norm) == 0.0 and float(scale) == 1.0 and norms.numel() == len(empty)


def test_norms_kept_do_not_hold_a_workspace():
    print("[norm] kept results", flush=True)
    gs = [torch.ones(1 << 22, device=dev()) for _ in range(16)]
    plan = om.GradNormPlan(gs)
    assert plan.ws_bytes > 8192
    out = plan.norm(gs, 1.0, per_tensor=True)
    assert all(t.untyped_storage().nbytes() == 4 * (2 + len(gs)) for t in out)
    assert out[0].item() == 2.0 ** 13 and bool((out[2] == 2.0 ** 11).all())


def test_grad_norm_range_and_specials():
    print("[norm] range", flush=True)
    for x in (1e-38, 1e-44, 1e-20, 1e20, 3e38):
        g = [torch.full((5000,), x, device=dev())]
        want = float(g[0][0].double()) * math.sqrt(5000)
        norm, scale = om.grad_norm(g, 1e-3)
        top = float(np.finfo(np.float32).max)
        # a subnormal result is rounded to a multiple of 2^-149
        assert (math.isinf(float(norm)) if want > top else
                abs(float(norm) - want) <= norm_bound(want) + 2.0 ** -150)
        expect = 1.0 if want <= 1e-3 else float(np.float32(1e-3)) / want
        assert abs(float(scale) - expect) <= 2 * E32 * expect + 2.0 ** -150
    for bad in (math.nan, math.inf, -math.inf):
        g = [torch.ones(70000, device=dev()), torch.ones(33, dtype=torch.bfloat16, device=dev())]
        g[1][32] = bad
        norm, scale, norms = om.GradNormPlan(g).norm(g, 1.0, per_tensor=True)
        assert math.isnan(float(scale)) and not math.isfinite(float(norm))
        assert abs(float(norms[0]) - math.sqrt(70000)) <= norm_bound(math.sqrt(70000))
    g = [torch.ones(50, device=dev()), torch.ones(40, device=dev())]
    plan = om.GradNormPlan(g)
    norm, _, norms = plan.norm([None, g[1]], per_tensor=True)             # left out: zero
    assert float(norms[0]) == 0.0 and abs(float(norm) - math.sqrt(40)) <= norm_bound(7.0)
    h = [g[0], g[0]]                                                      # the same one twice
    assert abs(float(om.grad_norm(h)[0]) - 10.0) <= norm_bound(10.0)


@pytest.mark.parametrize("gdt", ["f32", "bf16"])
def test_scale_in_place(gdt):
    print(f"[norm] in place {gdt}", flush=True)
    r = np.random.default_rng(2)
    gs = [on(r.normal(0, 1, n), DT[gdt]) for n in SIZES + [4 * 4096 + 5]]
    plan = om.GradNormPlan(gs)
    for value in (0.3, 1.0, 0.0, math.nan):
        was = [g.clone() for g in gs]
        plan.scale_(gs, on(value, torch.float32))
        torch.cuda.synchronize()
        for g, w in zip(gs, was):
            want = (w.float() * torch.tensor(value, device=dev())).to(DT[gdt]) if value != 1.0 else w
            assert torch.equal(torch.nan_to_num(g, 7.0), torch.nan_to_num(want, 7.0))
    before = [torch.zeros_like(g) for g in gs]
    plan.scale_(before[:-1] + [None], on(2.0, torch.float32))
    ps = [torch.nn.Parameter(torch.zeros(n, dtype=DT[gdt], device=dev())) for n in (5, 700, 9)]
    for p in ps[:2]:
        p.grad = on(r.normal(0, 1, p.numel()), DT[gdt])
    was = [f64(p.grad) for p in ps[:2]]
    want, factor, _ = oa.grad_norm(was, 0.25)
    norm = om.clip_grad_norm_(ps, 0.25)
    assert abs(float(norm) - want) <= norm_bound(want) and ps[2].grad is None
    half = 2.0 ** -8 if gdt == "bf16" else E32
    for p, w in zip(ps[:2], was):
        assert np.all(np.abs(f64(p.grad) - factor * w) <= (half + 4 * E32) * np.abs(factor * w))


# ---- streams, graphs, the front end ----------------------------------------------------------

@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
def test_on_another_stream(small):
    print(f"[adamw] stream small={small}", flush=True)
    s = Set([5, 70001], "bf16", "bf16", True, small)
    g = s.grads()
    norms = om.GradNormPlan(g)
    side = torch.cuda.Stream()
    prev = [s.before(i) for i in range(2)]
    cfg = om.make_adamw_config(step=1)
    side.wait_stream(torch.cuda.current_stream())
    norm, scale = norms.norm(g, 0.5, stream=side)
    s.plan.step(g, cfg, grad_scale=scale, stream=side)
    side.synchronize()
    for i in range(2):
        s.check(i, prev[i], g[i], cfg, float(scale), "stream")
    with torch.cuda.stream(side):
        again = norms.norm(g, 0.5)
    side.synchronize()
    assert torch.equal(again[0], norm)
    # a plan that is dropped while its step is still to run on the other stream
    t = Set([300001], "bf16", "bf16", True, small, seed=2)
    h, prev = t.grads(), [t.before(0)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(200):
            norms.norm(g, 0.5)                       # keeps the stream busy
    t.plan.step(h, cfg, stream=side)
    t.plan.close()
    t.plan = None
    junk = [torch.full((4096,), 255, dtype=torch.uint8, device=dev()) for _ in range(64)]
    side.synchronize()
    t.check(0, prev[0], h[0], cfg, label="dropped plan")
    del junk


@pytest.mark.parametrize("small", [False, True], ids=["f32", "8bit"])
def test_graph_replays_equal_eager_steps(small):
    """Norm and step captured together, replayed five times between eager work and
    synchronisations; every replay equals the eager run bitwise. Two graphs of one plan."""
    print(f"[adamw] graph small={small}", flush=True)
    def fresh():
        s = Set([300, 4097, 70001], "bf16", "bf16", True, small, seed=12)
        return s, s.grads()
    cfg = om.make_adamw_config(1e-2, step=5, seed=6, skip_nonfinite=True)
    s, g = fresh()
    norms = om.GradNormPlan(g)
    refs = []
    for k in range(6):
        norm, scale = norms.norm(g, 0.7)
        s.plan.step(g, cfg, grad_scale=scale)
        refs.append(s.bytes())
    t, h = fresh()
    norms2 = om.GradNormPlan(h)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            n2, s2 = norms2.norm(h, 0.7)
            t.plan.step(h, cfg, grad_scale=s2)
        graphs.append((graph, n2))
    for k in range(6):
        graphs[k % 2][0].replay()
        other = [x * 2 for x in g]                       # eager work between the replays
        om.grad_norm(other)
        torch.cuda.synchronize()
        assert all(np.array_equal(a, b) for a, b in zip(refs[k], t.bytes())), k
        assert torch.equal(graphs[k % 2][1], norm)


@pytest.mark.parametrize("state_bits,master", [(32, False), (32, True), (8, False), (8, True)])
def test_optimizer_steps_match_the_plan(state_bits, master):
    """The front end over two groups, clipped across both, a parameter whose gradient comes
    late, and a round trip through state_dict in the middle: each step against the oracle from
    the state before it."""
    print(f"[adamw] class state_bits={state_bits} master={master}", flush=True)
    r = np.random.default_rng(13)
    shapes = [(300, 17), (5,), (2, 3, 129), (513,)]
    ps = [torch.nn.Parameter(on(r.normal(0, 0.5, s), torch.bfloat16 if i < 2 else torch.float32))
          for i, s in enumerate(shapes)]
    groups = [{"params": ps[:2], "weight_decay": 0.2}, {"params": ps[2:], "wd_mul": 0.0, "lr": 3e-3}]
    make = lambda: om.AdamW(groups, lr=1e-2, betas=(0.9, 0.99), state_bits=state_bits,  # noqa: E731
                            master_weights=master, max_grad_norm=1.5, seed=3)
    opt = make()
    for k in range(1, 5):
        if k == 3:
            saved = opt.state_dict()
            groups = [{**g, "params": g["params"]} for g in groups]
            opt = make()
            opt.load_state_dict(saved)
        live = [0, 1, 2] if k == 1 else [0, 1, 2, 3]
        for i in range(4):
            ps[i].grad = on(r.normal(0, 1, shapes[i]), ps[i].dtype) if i in live else None
        grads = [f64(ps[i].grad) for i in live]
        norm, scale, _ = oa.grad_norm(grads, float(np.float32(1.5)))
        prev = {i: {q: (x.clone() if torch.is_tensor(x) else x) for q, x in opt.state[ps[i]].items()}
                for i in live}
        p_was = [p.detach().clone() for p in ps]
        opt.step()
        torch.cuda.synchronize()
        assert abs(float(opt.last_grad_norm) - norm) <= norm_bound(norm)
        for i in live:
            st, pv = opt.state[ps[i]], prev[i]
            t = st["step"]
            assert t == pv.get("step", 0) + 1
            n = ps[i].numel()
            lr, wd = (0.01, 0.2) if i < 2 else (0.003, 0.0)
            c = om.make_adamw_config(lr, (0.9, 0.99), 1e-8, wd, t)
            src = pv["master"] if "master" in pv else p_was[i]
            has = "exp_avg" in pv
            if state_bits == 8 and has:
                m0, r0 = (oa.held(adamw_ref.e4m3_values(adamw_ref.rows(u8(pv[k]), np.uint8)),
                                  adamw_ref.scale_values(u8(pv[k + "_scale"])), n)
                          for k in ("exp_avg", "exp_avg_sq"))
                v0 = r0 ** 2
            else:
                m0, v0 = ((f64(pv["exp_avg"]), f64(pv["exp_avg_sq"])) if has else
                          (np.zeros(n), np.zeros(n)))
            want, m, v = oa.adamw_step(f64(src), f64(ps[i].grad), m0, v0, t, c.lr, c.beta1, c.beta2,
                                       c.eps, c.weight_decay, scale)
            got = f64(st["master"]) if "master" in st else f64(ps[i])
            half = 2.0 ** -8 if ps[i].dtype == torch.bfloat16 and "master" not in st else 0.0
            # u is at most 10 for these betas, and off by at most 40 roundings of it
            assert np.all(np.abs(got - want) <= (half + 2 * E32) * np.abs(want) + c.lr * 400 * E32)
            if "master" in st:
                assert torch.equal(ps[i].detach(), st["master"].to(torch.bfloat16))
    assert ("master" in opt.state[ps[0]]) == master and "master" not in opt.state[ps[3]]
    if master:
        with torch.no_grad():
            ps[0].fill_(0.25)
        opt.refresh_masters()
        assert bool((opt.state[ps[0]]["master"] == 0.25).all())


def test_optimizer_without_clipping_matches_torch():
    """fp32 states and parameters against PyTorch's own AdamW over ten steps: both within
    rounding of the same trajectory (1e-5 of a parameter's movement per step)."""
    print("[adamw] torch AdamW", flush=True)
    r = np.random.default_rng(14)
    x0 = r.normal(0, 1, 3000)
    a = torch.nn.Parameter(on(x0, torch.float32))
    b = torch.nn.Parameter(on(x0, torch.float32))
    hyper = dict(lr=float(np.float32(1e-2)), betas=(float(np.float32(0.9)), float(np.float32(0.999))),
                 eps=float(np.float32(1e-8)), weight_decay=float(np.float32(0.1)))
    mine, theirs = om.AdamW([a], **hyper), torch.optim.AdamW([b], foreach=False, **hyper)
    for _ in range(10):
        g = on(r.normal(0, 1, 3000), torch.float32)
        a.grad, b.grad = g, g.clone()
        mine.step()
        theirs.step()
    assert float((a - b).detach().abs().max()) <= 10 * 1e-2 * 1e-5 + 20 * E32 * float(b.detach().abs().max())


@pytest.mark.parametrize("state_bits", [32, 8])
def test_first_step_under_capture_is_refused(state_bits):
    """...before a state is made: its zeros would be the graph's work, not done yet."""
    print(f"[adamw] first step captured, {state_bits} bits", flush=True)
    p = torch.nn.Parameter(torch.ones(700, device=dev()))
    p.grad = torch.ones(700, device=dev())
    opt = om.AdamW([p], state_bits=state_bits, max_grad_norm=1.0)
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            opt.step()
    assert not opt.state
    opt.step()
    other = torch.nn.Parameter(torch.ones(700, device=dev()))
    other.grad = p.grad
    om.AdamW([other], state_bits=state_bits, max_grad_norm=1.0).step()
    assert torch.equal(p.detach(), other.detach()) and bool((p.detach() < 1).all())


@pytest.mark.parametrize("state_bits", [32, 8])
def test_graph_outlives_its_plan_in_the_optimizer(state_bits):
    """A captured step replays after the optimizer has gone over to other gradients, and after a
    state was loaded: the tables and states that it was captured with are still there."""
    print(f"[adamw] graph and other gradients, {state_bits} bits", flush=True)
    r = np.random.default_rng(16)
    ps = [torch.nn.Parameter(on(r.normal(0, 1, n), torch.float32)) for n in (700, 5000)]
    gs = [on(r.normal(0, 1, p.numel()), torch.float32) for p in ps]
    opt = om.AdamW(ps, state_bits=state_bits, max_grad_norm=1.0)

    def step(grads):
        for p, g in zip(ps, grads):
            p.grad = g
        opt.step()

    step(gs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(gs)
    first = opt._plans[0][0]
    assert first.captured
    step([gs[0], None])                                        # another plan
    assert opt._plans[0][0] is not first and not opt._plans[0][0].captured
    assert opt._captured == [first] and first.handle and first._table is not None
    held = [[t.clone() for t in st.values() if torch.is_tensor(t)] for st in opt.state.values()]
    was = [p.detach().clone() for p in ps]
    junk = [torch.full((256,), 255, dtype=torch.uint8, device=dev()) for _ in range(64)]
    results = []
    for _ in range(3):                                         # from the same start each time
        with torch.no_grad():
            for p, w, st, h in zip(ps, was, opt.state.values(), held):
                p.copy_(w)
                for t, x in zip([t for t in st.values() if torch.is_tensor(t)], h):
                    t.view(torch.uint8).copy_(x.view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        results.append([p.detach().clone() for p in ps])
    for res in results:
        assert all(torch.equal(a, b) and not torch.equal(a, w)
                   for a, b, w in zip(res, results[0], was))
    opt.load_state_dict(opt.state_dict())
    assert first in opt._captured and not opt._plans
    graph.replay()                                             # on the states before the load
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(p.detach()).all()) for p in ps)
    assert copy.deepcopy(opt)._captured == []
    del junk


@pytest.mark.parametrize("state_bits", [32, 8])
def test_states_changed_from_outside(state_bits):
    """A step uses the states that the optimizer holds: after they were replaced by copies, moved
    to the host and back, or cleared. Against an optimizer whose states changed in place."""
    print(f"[adamw] states from outside, {state_bits} bits", flush=True)
    r = np.random.default_rng(17)
    sizes = (300, 5, 4097)
    x = [on(r.normal(0, 1, n), torch.bfloat16) for n in sizes]
    sets = [[torch.nn.Parameter(t.clone()) for t in x] for _ in range(2)]
    opts = [om.AdamW([{"params": ps[:2]}, {"params": ps[2:], "lr": 1e-2}], state_bits=state_bits,
                     master_weights=True, weight_decay=0.1) for ps in sets]
    mine, other = opts

    def step():
        gs = [on(r.normal(0, 1, n), torch.bfloat16) for n in sizes]
        for ps, opt in zip(sets, opts):
            for p, g in zip(ps, gs):
                p.grad = g.clone()
            opt.step()
        torch.cuda.synchronize()
        for a, b in zip(*sets):
            assert torch.equal(a.detach(), b.detach())
            assert mine.state[a].keys() == other.state[b].keys()
            for k, t in mine.state[a].items():
                assert (torch.equal(t.view(torch.uint8), other.state[b][k].view(torch.uint8))
                        if torch.is_tensor(t) else t == other.state[b][k]), k

    step()
    step()
    plans = [opt._plans[0][0] for opt in opts]
    step()
    assert all(opt._plans[0][0] is plan for opt, plan in zip(opts, plans))     # as long as they fit
    for st in mine.state.values():                     # the same values in other tensors
        for k, t in st.items():
            if torch.is_tensor(t):
                st[k] = t.cpu().to(dev())
    step()
    mine.state[sets[0][2]] = dict(mine.state[sets[0][2]])                      # another dict
    step()
    mine.state[sets[0][2]]["exp_avg"] = torch.zeros_like(mine.state[sets[0][2]]["exp_avg"])
    other.state[sets[1][2]]["exp_avg"].view(torch.uint8).zero_()
    step()
    mine.state.clear()                                 # as before the first step
    for p, st in other.state.items():
        for k, t in st.items():
            if torch.is_tensor(t):
                t.copy_(p.detach()) if k == "master" else t.view(torch.uint8).zero_()
        st["step"] = 0
    step()
    mine.state[sets[0][0]]["exp_avg"] = mine.state[sets[0][0]]["exp_avg"].cpu()
    with pytest.raises(ValueError):
        mine.step()


def test_skipped_steps_of_the_optimizer():
    print("[adamw] optimizer skip", flush=True)
    p = torch.nn.Parameter(torch.ones(1000, device=dev()))
    opt = om.AdamW([p], max_grad_norm=1.0, skip_nonfinite=True, state_bits=8)
    p.grad = torch.ones(1000, device=dev())
    opt.step()
    was, m = p.detach().clone(), opt.state[p]["exp_avg"].view(torch.uint8).clone()
    p.grad = torch.full((1000,), math.inf, device=dev())
    opt.step()
    assert torch.equal(p.detach(), was) and torch.equal(opt.state[p]["exp_avg"].view(torch.uint8), m)
    assert math.isinf(float(opt.last_grad_norm))
    p.grad = torch.ones(1000, device=dev())
    opt.step()
    assert bool((p.detach() < was).all())


def test_skipping_without_clipping():
    print("[adamw] skip without clipping", flush=True)
    ps = [torch.nn.Parameter(torch.ones(700, device=dev())) for _ in range(2)]
    opt = om.AdamW([{"params": ps[:1]}, {"params": ps[1:], "state_bits": 8}], skip_nonfinite=True)
    for p in ps:
        p.grad = torch.full((700,), 100.0, device=dev())
    opt.step()
    was = [p.detach().clone() for p in ps]
    assert all(bool((p.detach() < 1).all()) for p in ps)           # a norm over 1 is not clipped
    ps[1].grad[3] = math.nan                                       # in one group: neither moves
    opt.step()
    assert all(torch.equal(p.detach(), w) for p, w in zip(ps, was))


def test_clipping_in_front_of_the_other_optimizers():
    """clip_grad_norm_ over all gradients, then Muon for the matrix and CautiousAdam for the
    rest: the same bits as those optimizers given the clipped gradients."""
    print("[norm] in front of Muon and CautiousAdam", flush=True)
    r = np.random.default_rng(15)
    outs = []
    for clipped in (True, False):
        r = np.random.default_rng(15)
        w = torch.nn.Parameter(on(r.normal(0, 0.02, (96, 160)), torch.bfloat16))
        b = torch.nn.Parameter(on(r.normal(0, 0.02, 777), torch.float32))
        w.grad, b.grad = on(r.normal(0, 1, (96, 160)), torch.bfloat16), on(r.normal(0, 1, 777), torch.float32)
        if clipped:
            om.clip_grad_norm_([w, b], 1.0)
        else:
            scale = om.grad_norm([w.grad, b.grad], 1.0)[1]
            w.grad, b.grad = (w.grad.float() * scale).to(torch.bfloat16), b.grad * scale
        om.Muon([w]).step()
        om.CautiousAdam([b]).step()
        torch.cuda.synchronize()
        outs.append((w.detach().clone(), b.detach().clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_refusals_with_device_tensors():
    p, m, v = (torch.zeros(300, device=dev()) for _ in "pmv")
    plan = om.AdamWPlan([p], [m], [v], [torch.float32])
    cfg = om.make_adamw_config()
    ok = torch.zeros(300, device=dev())
    for bad in ([], [ok, ok], [ok[:299]], [ok.bfloat16()], [ok.cpu()], [torch.zeros(600, device=dev())[::2]]):
        with pytest.raises((ValueError, TypeError)):
            plan.step(bad, cfg)
    with pytest.raises(om.MuonError):
        plan.step([p], cfg)                                               # the parameter itself
    with pytest.raises(om.MuonError):
        plan.step([torch.zeros(301, device=dev())[1:]], cfg)              # 4-byte aligned
    with pytest.raises(ValueError, match="memory"):
        plan.step([torch._neg_view(ok)], cfg)                             # its memory: other values
    for scale in (torch.ones(2, device=dev()), torch.ones(1), torch.ones(1, device=dev()).half()):
        with pytest.raises(ValueError):
            plan.step([ok], cfg, grad_scale=scale)
    with pytest.raises(om.MuonError):
        om.AdamWPlan([p], [m], [m], [torch.float32])                      # one buffer twice
    with pytest.raises(om.MuonError):
        om.GradNormPlan([ok]).norm([ok], -1.0)
    with pytest.raises(om.MuonError):
        om.GradNormPlan([ok, ok]).scale_([ok, ok], torch.ones(1, device=dev()))
    assert not bool(p.any() or m.any() or v.any())
