"""Host-side tests of include/mx4.h and include/orthogonalize.h: sizes, validation (which comes before any
launch, so that these run without a GPU on addresses that are never read), a C99 caller, and the Python
wrappers' refusals. The product kernels' reads of LDS are checked in the compiled code."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import asm_check
import orthogonalized_momentum_optimizer_amd as om
from orthogonalized_momentum_optimizer_amd import _lib as L
from orthogonalized_momentum_optimizer_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "orthogonalized_momentum_optimizer_amd")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
OK, INV, UNSUP, WS = 0, -1, -2, -3
BASE = 1 << 40
HUGE = 2 ** 64 - 1
MAX_SIDE = 2 ** 31 - 256

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake device addresses are only used without a GPU")


def status_of(f, *args):
    try:
        f(*args)
    except om.MuonError as e:
        return e.status
    return OK


@pytest.mark.parametrize("rows,cols,tiles", [(0, 5, 0), (5, 0, 0), (1, 1, 1), (16, 128, 1), (17, 128, 2), (16, 129, 2),
                                             (33, 257, 9), (333, 777, 21 * 7), (16384, 6400, 1024 * 50)])
def test_sizes_of_held_values(rows, cols, tiles):
    assert L.muon_mx_codes_size(rows, cols) == tiles * 1024
    assert L.muon_mx_scales_size(rows, cols) == tiles * 64


@pytest.mark.parametrize("rows,cols", [(-1, 4), (4, -1), (MAX_SIDE + 1, 1), (1, MAX_SIDE + 1), (1 << 21, 1 << 20)])
def test_sizes_outside_the_limits(rows, cols):
    assert L.muon_mx_codes_size(rows, cols) == HUGE and L.muon_mx_scales_size(rows, cols) == HUGE
    assert L.muon_mx_matmul_workspace_size(rows, 1, cols) == HUGE
    assert L.muon_mx_matmul_workspace_size(1, rows, cols) == HUGE


def test_product_workspace():
    assert L.muon_mx_matmul_workspace_size(0, 5, 5) == 0
    assert L.muon_mx_matmul_workspace_size(16384, 6400, 1600) == 0      # enough tiles
    need = L.muon_mx_matmul_workspace_size(128, 128, 1 << 20)           # one tile of a long sum: split
    assert need > 0 and need % (128 * 128 * 4) == 0


def source(**kw):
    s = dict(x=BASE, rows=20, cols=40, row_stride=40, dtype=1, codes=BASE + (1 << 20), scales=BASE + (2 << 20),
             codes_t=BASE + (3 << 20), scales_t=BASE + (4 << 20))
    s.update(kw)
    return tuple(s[k] for k in ("x", "rows", "cols", "row_stride", "dtype", "codes", "scales", "codes_t",
                                "scales_t"))


def quantize(*entries, n=None, stochastic=0):
    a = L.make_mx_sources(entries)
    return status_of(L.muon_mx_quantize, a, len(entries) if n is None else n, stochastic, 0, None)


BAD_SOURCES = [
    (dict(dtype=7), INV), (dict(rows=-1), INV), (dict(cols=-1), INV), (dict(rows=MAX_SIDE + 1), UNSUP),
    (dict(rows=1 << 20, cols=(1 << 20) + 1), UNSUP), (dict(scales=None), INV), (dict(codes=None), INV),
    (dict(scales_t=None), INV), (dict(codes=None, scales=None, codes_t=None, scales_t=None), INV),
    (dict(x=None), INV), (dict(x=BASE + 2), INV), (dict(dtype=0, x=BASE + 1), INV), (dict(row_stride=39), INV),
    (dict(row_stride=-40), INV), (dict(codes=BASE + (1 << 20) + 8), INV), (dict(scales_t=BASE + 8), INV),
    (dict(codes=BASE), INV),                                             # over its source
    (dict(codes=BASE + 20 * 40 * 4 - 16), INV),
    (dict(scales=BASE + (1 << 20) + 1024), INV),                         # over its own codes (2 KB)
    (dict(codes_t=BASE + (1 << 20)), INV),
    (dict(rows=1 << 31, cols=1), UNSUP),
]


@no_gpu_only
@pytest.mark.parametrize("change,want", BAD_SOURCES)
def test_quantize_refuses(change, want):
    assert quantize(source(**change)) == want
    assert quantize(source(x=BASE + (8 << 20), codes=BASE + (9 << 20), scales=BASE + (10 << 20), codes_t=None,
                           scales_t=None), source(**change)) == want


@no_gpu_only
def test_quantize_lists():
    assert quantize(n=0) == OK
    assert status_of(L.muon_mx_quantize, None, 0, 0, 0, None) == OK
    assert status_of(L.muon_mx_quantize, None, 1, 0, 0, None) == INV
    assert quantize(source(), n=-1) == INV
    assert quantize(source(), stochastic=2) == INV
    assert quantize(source(), source()) == INV                           # the same results twice
    assert quantize(source(rows=0, x=None), source(cols=0, x=None)) == OK
    # a result over another source
    assert quantize(source(), source(x=BASE + (1 << 20), codes=BASE + (9 << 20), scales=BASE + (10 << 20),
                                     codes_t=None, scales_t=None)) == INV


@no_gpu_only
@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), INV), (dict(rows=-1), INV), (dict(cols=MAX_SIDE + 1), UNSUP), (dict(codes=None), INV),
    (dict(scales=None), INV), (dict(codes=BASE + 4), INV), (dict(out=None), INV), (dict(out=BASE + 2 + (1 << 30)), INV),
    (dict(out=BASE), INV), (dict(out=BASE + (1 << 20) - 4), INV), (dict(rows=1 << 25, cols=1 << 14), UNSUP),
    (dict(rows=0, codes=None, out=None), OK), (dict(cols=0, scales=None, out=None), OK)])
def test_dequantize_refuses(change, want):
    a = dict(codes=BASE, scales=BASE + (1 << 20), rows=20, cols=40, out=BASE + (1 << 30), dtype=1)
    a.update(change)
    assert status_of(L.muon_mx_dequantize, a["codes"], a["scales"], a["rows"], a["cols"], a["out"], a["dtype"],
                     None) == want


@no_gpu_only
@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), INV), (dict(m=-1), INV), (dict(n=-1), INV), (dict(k=-1), INV), (dict(m=MAX_SIDE + 1), UNSUP),
    (dict(m=1 << 20, n=1 << 20), UNSUP), (dict(out=None), INV), (dict(out=BASE + (1 << 31) + 2), INV),
    (dict(ac=None), INV), (dict(bs=None), INV), (dict(bc=BASE + 8), INV), (dict(out=BASE), INV),
    (dict(out=BASE + (3 << 20)), INV), (dict(m=128, n=128, k=1 << 20), WS),
    (dict(m=128, n=128, k=1 << 20, ws=BASE + (1 << 32), bytes=64), WS),
    (dict(m=128, n=128, k=1 << 20, ws=BASE + (1 << 32) + 8, bytes=1 << 31), WS),
    (dict(m=128, n=128, k=1 << 20, ws=BASE + (1 << 31), bytes=1 << 31), INV),     # over out
    (dict(m=0, out=None, ac=None), OK), (dict(n=0, out=None), OK)])
def test_matmul_refuses(change, want):
    a = dict(ac=BASE, **{"as": BASE + (1 << 28)}, bc=BASE + (2 << 28), bs=BASE + (3 << 28), m=20, n=30, k=40,
             out=BASE + (1 << 31), dtype=1, ws=None, bytes=0)
    if "k" not in change:
        a.update({"as": BASE + (1 << 20), "bc": BASE + (2 << 20), "bs": BASE + (3 << 20)})
    a.update(change)
    assert status_of(L.muon_mx_matmul, a["ac"], a["as"], a["bc"], a["bs"], a["m"], a["n"], a["k"], a["out"],
                     a["dtype"], a["ws"], a["bytes"], None) == want


# ---- orthogonalize.h ---------------------------------------------------------------------------

def test_orthogonalize_workspace():
    size = L.muon_orthogonalize_workspace_size
    assert size(1, 0, 4, 4) == size(0, 1, 4, 4) == size(1, 1, 0, 4) == size(1, 1, 4, 0) == 0
    assert size(1, 1200, 64, 1600) == 0                                  # in one launch
    assert 0 < size(1, 300, 128, 1024) < 1 << 29 and size(1, 300, 128, 1024) % 256 == 0
    assert 0 < size(1, 12, 64, 8192) < 1 << 29
    assert size(1, 1 << 20, 128, 128) < 1 << 30                          # in batches
    for bad in [(1, 1, 129, 129), (1, 1, 1, (1 << 24) + 1), (1 << 13, 1 << 12, 4, 4), (-1, 1, 4, 4), (1, 1, -4, 4)]:
        assert size(*bad) == HUGE


def orth(cfg=(), ws=None, bytes_=0, **kw):
    s = dict(in_=BASE, out=BASE + (1 << 30), outer=1, inner=3, rows=8, cols=40, in_stride=(0, 320, 40, 1),
             out_stride=(0, 320, 40, 1), dtype=1)
    s.update(kw)
    k = L.muon_stack()
    for name, v in s.items():
        if name.endswith("stride"):
            for i, e in enumerate(v):
                getattr(k, name)[i] = e
        else:
            setattr(k, name, v)
    c = L.muon_config_default()
    for name, v in cfg:
        setattr(c, name, v)
    return status_of(L.muon_orthogonalize, k, c, ws, bytes_, None)


WIDE = dict(outer=1, inner=3, rows=128, cols=200, in_stride=(0, 25600, 200, 1), out_stride=(0, 25600, 200, 1))


@no_gpu_only
@pytest.mark.parametrize("kw,want", [
    (dict(dtype=5), INV), (dict(rows=-1), INV), (dict(rows=129, cols=129), UNSUP), (dict(inner=1 << 25), UNSUP),
    (dict(in_=None), INV), (dict(out=None), INV), (dict(in_=BASE + 2), INV), (dict(out=BASE + (1 << 30) + 1), INV),
    (dict(in_stride=(0, 320, 40, 2)), INV), (dict(in_stride=(0, 320, 1, 8)), INV),      # not the same side
    (dict(in_stride=(0, -320, 40, 1)), INV), (dict(in_stride=(0, 1 << 41, 40, 1)), INV),
    (dict(out_stride=(0, 0, 40, 1)), INV), (dict(out_stride=(0, 320, 39, 1)), INV),
    (dict(out_stride=(0, 160, 40, 1)), INV), (dict(out=BASE + 4), INV), (dict(out=BASE, out_stride=(0, 400, 40, 1)), INV),
    (dict(inner=0, in_=None), OK), (dict(cols=0, in_=None), OK),
    (dict(cfg=[("ns_steps", -1)]), INV), (dict(cfg=[("eps", float("nan"))]), INV), (dict(cfg=[("eps", -1.0)]), INV),
    (dict(cfg=[("a", float("inf"))]), INV),
    (dict(WIDE), WS), (dict(WIDE, ws=BASE + (1 << 32), bytes_=256), WS),
    (dict(WIDE, ws=BASE + (1 << 32) + 128, bytes_=1 << 31), WS), (dict(WIDE, ws=BASE + (1 << 30), bytes_=1 << 31), INV)])
def test_orthogonalize_refuses(kw, want):
    assert orth(**kw) == want


@no_gpu_only
def test_orthogonalize_refuses_null():
    c = L.muon_config_default()
    assert L.lib().muon_orthogonalize(None, ctypes.byref(c), None, 0, None) == INV
    assert L.lib().muon_orthogonalize(ctypes.byref(L.muon_stack()), None, None, 0, None) == INV


# ---- the wrappers without a GPU ------------------------------------------------------------------

def test_wrappers_refuse_cpu_tensors():
    x, w = torch.randn(4, 8), torch.randn(6, 8)
    for call in (lambda: om.mx4_quantize(x), lambda: om.mx4_quantize_both(x), lambda: om.mx4_linear(x, w),
                 lambda: om.orthogonalize(x), lambda: om.MX4Copies([w])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        om.mx4_linear(x, [w])
    with pytest.raises(TypeError):
        om.mx4_linear(x.double(), w)
    with pytest.raises(ValueError):
        om.mx4_linear(x, w[:, :4])
    with pytest.raises(TypeError):
        om.mx4_matmul(x, w)
    with pytest.raises(TypeError):
        om.MX4Copies([1])
    assert len(om.MX4Copies([])) == 0


# ---- a C caller, and the compiled code -------------------------------------------------------------

@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc is not available")
def test_c_program_uses_the_abi(tmp_path):
    exe = str(tmp_path / "mx4_check")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(ROCM, "include"),
                        os.path.join(ROOT, "tests", "c_abi", "mx4_check.c"), "-o", exe, "-L", PKG, "-lmuon",
                        "-Wl,-rpath," + PKG, "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
                        "-Wl,-rpath," + os.path.join(ROCM, "lib")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=dict(os.environ, HIP_VISIBLE_DEVICES=""))
    assert r.returncode == 0, r.stdout + r.stderr
    assert "abi ok" in r.stdout


@pytest.mark.parametrize("src", ["mx4_matmul.hip", "mx4_quantize.hip"])
def test_no_use_of_lds_read_results_before_their_wait(src):
    try:
        path = build.device_asm(src)
    except RuntimeError as e:  # no HIP toolchain on this host
        pytest.skip(str(e))
    text = open(path).read()
    assert "ds_read" in text
    v = asm_check.violations(text)
    assert not v, "\n".join(v[:10])
