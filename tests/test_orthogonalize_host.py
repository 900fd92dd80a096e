"""Host-side tests of the passes of include/orthogonalize.h (validation comes before any HIP call)."""
import ctypes

import pytest

import orthogonalized_momentum_optimizer_amd as om
from orthogonalized_momentum_optimizer_amd import _lib as L

INV, UNS = -1, -2
DEFAULT = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("abc,steps,want", [
    (DEFAULT, 0, 1), (DEFAULT, 1, 1), (DEFAULT, 5, 1), (DEFAULT, 8, 1), (DEFAULT, 9, 2), (DEFAULT, 16, 2),
    (DEFAULT, 17, 3), (DEFAULT, 64, 8), ((2.0, -1.5, 0.5), 15, 1), ((2.0, -1.5, 0.5), 16, 2),
    ((1.5, -0.5, 0.0), 25, 1), ((1.5, -0.5, 0.0), 26, 2), ((1.0, 0.0, 0.0), 64, 1), ((0.5, 0.0, 0.0), 64, 1),
    ((1e30, 0.0, 0.0), 3, 3), ((-3.4445, 4.7750, -2.0315), 9, 2), ((1.0, 1.0, 0.0), 2, 1),
    # q(x) = 1 + x on [0, 1], then A up to 4 and X lifted by 5: 2 * 5 = 10, and A up to 100: 101, A 1e6: past 2^15
    ((1.0, 1.0, 0.0), 3, 1), ((1.0, 1.0, 0.0), 4, 2)])
def test_passes_follow_what_rounds_can_lift(abc, steps, want):
    assert L.muon_orthogonalize_passes(om.make_config(ns_steps=steps, abc=abc)) == want


def test_a_schedule_counts_its_largest_run():
    """Rounds that shrink everything do not pay for those that lift."""
    up, down = (16.0, 0.0, 0.0), (1 / 16, 0.0, 0.0)
    passes = lambda s: L.muon_orthogonalize_passes(om.make_config(ns_steps=len(s), schedule=s))  # noqa: E731
    assert passes([up] * 3) == 1 and passes([up] * 4) == 2
    assert passes([down] * 9 + [up] * 3) == 1 and passes([down] * 9 + [up] * 4) == 2
    assert passes([up, down] * 9) == 1


def test_passes_refuse_bad_rounds():
    bad = om.make_config(ns_steps=5)
    bad.ns_steps = 65
    with pytest.raises(om.MuonError):
        L.muon_orthogonalize_passes(bad)
    assert L.lib().muon_orthogonalize_passes(None) == INV


def test_bf16_stacks_of_several_passes_are_refused():
    k = L.muon_stack(in_=1 << 40, out=1 << 41, outer=1, inner=2, rows=4, cols=8, dtype=0)
    k.in_stride = k.out_stride = (ctypes.c_int64 * 4)(0, 32, 8, 1)
    cfg = om.make_config(ns_steps=9)
    assert L.lib().muon_orthogonalize(ctypes.byref(k), ctypes.byref(cfg), None, 0, None) == UNS
    assert "fp32" in L.muon_last_error()
