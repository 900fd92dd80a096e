"""8-bit states at the top of fp32's range: what is held there decodes to values that the next
step can use, and a block comes back from them. Byte by byte against the fp32 evaluation of
adamw_ref.py, whose codes beyond the largest ones held are replaced by these."""
import numpy as np
import pytest
import torch

import adamw_ref
import orthogonalized_momentum_optimizer_amd as om
from test_gpu_adamw import DT, Set, f64, u8

pytestmark = pytest.mark.gpu

CODE_240 = 0x77                                  # 1.875 2^7
MEAN_SCALE = 120 + 127                           # of a block with an |m| of 1.77 2^127 or more
ROOT_SCALE = 56 + 127                            # of a block with an r of 1.77 2^63 or more


def held(codes, scales, top_scale):
    """Codes whose value is over 240 times the largest scale, NaN apart, as +-240."""
    over = (np.repeat(scales, 256)[:codes.size] == top_scale) & ((codes & 0x7f) > CODE_240) & (
        (codes & 0x7f) != 0x7f)
    return np.where(over, (codes & 0x80) | CODE_240, codes).astype(np.uint8)


def step_and_compare(s, cfg, grads, label):
    prev = [s.before(i) for i in range(len(s.sizes))]
    s.plan.step(grads, cfg)
    torch.cuda.synchronize()
    for i, g in enumerate(grads):
        _, mc, ms, rc, rs = prev[i]
        want = adamw_ref.step_codes(f64(g).astype(np.float32), mc, ms, rc, rs, cfg.beta1, cfg.beta2,
                                    cfg.seed, cfg.step, cfg.stochastic)
        got = (u8(s.m[i]), u8(s.ms[i]), u8(s.v[i]), u8(s.vs[i]))
        want = (held(want[0], want[1], MEAN_SCALE), want[1], held(want[2], want[3], ROOT_SCALE), want[3])
        for name, a, b in zip(("m", "m scale", "r", "r scale"), got, want):
            assert np.array_equal(a, b), f"{label} tensor {i}: {name}"


def roots(s, i):
    return adamw_ref.e4m3_values(u8(s.v[i])) * np.repeat(adamw_ref.scale_values(u8(s.vs[i])), 256)[
        :s.sizes[i]].astype(np.float32)


@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_block_comes_back_from_a_v_at_the_top(dt, stochastic):
    """One v beyond fp32's range, or at its end: its square stays finite, and 140 steps of beta2 =
    0.5 later (r falls by 0.71 a step, 2^64 to 2^-6) the block holds what its gradients give."""
    print(f"[adamw range] v {dt} stochastic={stochastic}", flush=True)
    # v = g^2 in the first step: infinite, 0.99 2^128, 0.90 2^128, 0.86 2^128 (below the largest)
    tops = [1e30] + [float(2.0 ** 64 * x ** 0.5) for x in (0.99, 0.90, 0.86)]
    s = Set([4096, 300], dt, dt, False, True, seed=8)
    for t in range(1, 142):
        g = s.grads()
        if t == 1:
            for k, x in enumerate(tops):
                g[0][256 * k + 5] = g[1][k] = x
        cfg = om.make_adamw_config(1e-3, (0.9, 0.0 if t == 1 else 0.5), step=t, seed=t,
                                   stochastic=stochastic)
        step_and_compare(s, cfg, g, f"step {t}")
        with np.errstate(over="ignore"):
            assert all(np.isfinite(roots(s, i) ** 2).all() for i in range(2))
        if t == 1:
            assert all(roots(s, 0)[256 * k + 5] == np.float32(240 * 2.0 ** 56) for k in range(3))
    # a root mean square of gradients of at most 5 (5 sigma of 1, 4396 values a step: 3e-7 each)
    assert all(roots(s, i).max() < 6 for i in range(2))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_finite_m_at_the_top_stays_finite(dt):
    """Without averaging m is the gradient: the largest ones, of either sign, leave a finite m and
    parameter, and the next gradient replaces them."""
    print(f"[adamw range] m {dt}", flush=True)
    s = Set([4096, 300], dt, dt, False, True, seed=9)
    top = torch.finfo(DT[dt]).max
    for t in (1, 2, 3):
        g = s.grads()
        if t == 1:
            for k, x in enumerate((top, -top, -top * 0.98, top * 0.95, top * 0.9)):
                g[0][256 * k + 9] = g[1][k] = x
        step_and_compare(s, om.make_adamw_config(1e-3, (0.0, 0.9), step=t, seed=t), g, f"step {t}")
        for i in range(2):
            m = s.m[i].float() * torch.repeat_interleave(s.ms[i].float(), 256)[:s.sizes[i]]
            assert bool(torch.isfinite(m).all()) and bool(torch.isfinite(s.p[i]).all())
            # e4m3 of an ordinary gradient (at most 6 sigma), or 240 / 256 of 2^128 and 2^-4 of it less
            assert float(m.abs().max()) < 7 if t > 1 else float(m.abs().max()) >= 0.93 * 2.0 ** 127.9
