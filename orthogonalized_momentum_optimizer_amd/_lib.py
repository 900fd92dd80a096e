"""ctypes binding of libmuon.so (the C ABI of the headers under include/), with the same names.

Only argument marshalling happens here: every step of the optimizer runs in the HIP
kernels of the library. PyTorch's HIP runtime is loaded first (``import torch``) so the
library binds to that same runtime and can use torch's device pointers and streams.
A missing or unloadable library is an error, never a fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Sequence

import torch  # noqa: F401  (loads the HIP runtime the library must share)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmuon.so")

MUON_OK = 0
MUON_ERR_INVALID_ARG = -1
MUON_ERR_UNSUPPORTED = -2
MUON_ERR_WORKSPACE = -3
MUON_ERR_HIP = -4

MUON_DT_BF16 = 0
MUON_DT_F32 = 1
MUON_NS_BF16 = 0
MUON_NS_F32_DEBUG = 1

KERNEL_KINDS = ("momentum", "norm", "gram", "poly", "apply", "update", "roweq", "rounds")

EXPORTED = (
    "muon_config_default", "muon_plan_create", "muon_plan_workspace_size", "muon_step",
    "muon_newton_schulz", "muon_plan_destroy", "muon_plan_set_profiling",
    "muon_plan_read_profile", "muon_status_string", "muon_last_error",
    "muon_adam_config_default", "muon_cautious_adam_step", "muon_step_noalloc",
    "muon_plan_set_concurrency", "muon_plan_set_fused",
    "muon_adamw_config_default", "muon_adamw_plan_create", "muon_adamw_step",
    "muon_adamw_check",
    "muon_adamw_plan_table_size", "muon_adamw_plan_upload",
    "muon_adamw_plan_destroy", "muon_grad_plan_create", "muon_grad_plan_workspace_size",
    "muon_grad_norm", "muon_grad_scale", "muon_grad_plan_destroy",
    "muon_mx_codes_size", "muon_mx_scales_size", "muon_mx_quantize", "muon_mx_dequantize",
    "muon_mx_matmul_workspace_size", "muon_mx_matmul",
    "muon_orthogonalize_workspace_size", "muon_orthogonalize_passes", "muon_orthogonalize",
)
MUON_MAX_STREAMS = 4
MUON_ADAMW_F32 = 0
MUON_ADAMW_8BIT = 1
MUON_ADAMW_BLOCK = 256
MUON_STATIC_SCRATCH_BYTES = 64 << 20


class MuonError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_string(status)}: {message}")
        self.status = status


class muon_matrix(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("momentum", ctypes.c_void_p),
        ("update_out", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("param_dtype", ctypes.c_int),
        ("grad_dtype", ctypes.c_int),
        ("row_var", ctypes.c_void_p),
    ]


class muon_config(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float),
        ("beta", ctypes.c_float),
        ("nesterov", ctypes.c_int),
        ("ns_steps", ctypes.c_int),
        ("a", ctypes.c_float),
        ("b", ctypes.c_float),
        ("c", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("schedule", ctypes.POINTER(ctypes.c_float)),
        ("row_equalize", ctypes.c_int),
        ("row_beta", ctypes.c_float),
        ("row_eps", ctypes.c_float),
    ]


class muon_adam_tensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("exp_avg", ctypes.c_void_p),
        ("exp_avg_sq", ctypes.c_void_p),
        ("numel", ctypes.c_int64),
        ("param_dtype", ctypes.c_int),
        ("grad_dtype", ctypes.c_int),
        ("wd_mul", ctypes.c_float),
    ]


class muon_adam_config(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float),
        ("beta1", ctypes.c_float),
        ("beta2", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("step", ctypes.c_int64),
    ]


class muon_adamw_tensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("master", ctypes.c_void_p),
        ("exp_avg", ctypes.c_void_p),
        ("exp_avg_sq", ctypes.c_void_p),
        ("exp_avg_scale", ctypes.c_void_p),
        ("exp_avg_sq_scale", ctypes.c_void_p),
        ("numel", ctypes.c_int64),
        ("param_dtype", ctypes.c_int),
        ("grad_dtype", ctypes.c_int),
        ("wd_mul", ctypes.c_float),
    ]


class muon_adamw_config(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float),
        ("beta1", ctypes.c_float),
        ("beta2", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("step", ctypes.c_int64),
        ("grad_scale", ctypes.c_void_p),
        ("skip_nonfinite", ctypes.c_int),
        ("stochastic", ctypes.c_int),
        ("seed", ctypes.c_uint64),
    ]


class muon_mx_source(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int),
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("codes_t", ctypes.c_void_p),
        ("scales_t", ctypes.c_void_p),
    ]


class muon_stack(ctypes.Structure):
    _fields_ = [
        ("in_", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("outer", ctypes.c_int64),
        ("inner", ctypes.c_int64),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("in_stride", ctypes.c_int64 * 4),
        ("out_stride", ctypes.c_int64 * 4),
        ("dtype", ctypes.c_int),
    ]


_lib = None
_args = None


def args():
    """The native part of the binding (csrc/tensor_args.cpp); raises if it has not been built."""
    global _args
    if _args is None:
        try:
            from . import _tensor_args
        except ImportError as e:
            raise RuntimeError("_tensor_args.so is missing: build it with `python -m "
                               "orthogonalized_momentum_optimizer_amd.build`") from e
        L = lib()
        _tensor_args.bind(*(address_of(f) for f in (
            L.muon_mx_quantize, L.muon_mx_dequantize, L.muon_mx_matmul,
            L.muon_mx_matmul_workspace_size, L.muon_orthogonalize,
            L.muon_orthogonalize_workspace_size, L.muon_orthogonalize_passes, L.muon_last_error)))
        _args = _tensor_args
    return _args


def tensor_addresses(tensors, numels, dtypes, device: int):
    """The addresses of a list of tensors (None: 0) as a ctypes array, or the index of the first
    one that is not a contiguous tensor of its ``numels`` and ``dtypes`` entry on ``device``.
    ``numels``, ``dtypes``: ctypes arrays of int64 and of muon_dtype as int32 (2: float8_e4m3fn,
    3: float8_e8m0fnu)."""
    out = (ctypes.c_void_p * len(numels))()
    bad = args().addresses(tensors, numels, dtypes, device, out)
    return out if bad < 0 else bad


def address_of(function) -> int:
    """The address of a function of the library."""
    return ctypes.cast(function, ctypes.c_void_p).value


def lib() -> ctypes.CDLL:
    """The loaded library; raises if libmuon.so has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m orthogonalized_momentum_optimizer_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    L.muon_config_default.argtypes = [ctypes.POINTER(muon_config)]
    L.muon_config_default.restype = None
    L.muon_plan_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(i64), ctypes.POINTER(i64),
                                   ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                                   i64, ctypes.c_int]
    L.muon_plan_create.restype = ctypes.c_int
    L.muon_plan_workspace_size.argtypes = [vp]
    L.muon_plan_workspace_size.restype = sz
    L.muon_step.argtypes = [vp, ctypes.POINTER(muon_matrix), i64, ctypes.POINTER(muon_config),
                            vp, sz, vp]
    L.muon_step.restype = ctypes.c_int
    L.muon_step_noalloc.argtypes = [vp, ctypes.POINTER(muon_matrix), i64,
                                    ctypes.POINTER(muon_config), ctypes.c_void_p]
    L.muon_step_noalloc.restype = ctypes.c_int
    L.muon_newton_schulz.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), i64,
                                     ctypes.POINTER(muon_config), vp, sz, vp]
    L.muon_newton_schulz.restype = ctypes.c_int
    L.muon_plan_destroy.argtypes = [vp]
    L.muon_plan_destroy.restype = None
    L.muon_plan_set_profiling.argtypes = [vp, ctypes.c_int]
    L.muon_plan_set_profiling.restype = ctypes.c_int
    L.muon_plan_set_concurrency.argtypes = [vp, ctypes.c_int]
    L.muon_plan_set_concurrency.restype = ctypes.c_int
    L.muon_plan_set_fused.argtypes = [vp, ctypes.c_int]
    L.muon_plan_set_fused.restype = ctypes.c_int
    L.muon_plan_read_profile.argtypes = [vp, ctypes.POINTER(ctypes.c_double),
                                         ctypes.POINTER(i64), ctypes.c_int]
    L.muon_plan_read_profile.restype = ctypes.c_int
    L.muon_adam_config_default.argtypes = [ctypes.POINTER(muon_adam_config)]
    L.muon_adam_config_default.restype = None
    L.muon_cautious_adam_step.argtypes = [ctypes.POINTER(muon_adam_tensor), i64,
                                          ctypes.POINTER(muon_adam_config), vp]
    L.muon_cautious_adam_step.restype = ctypes.c_int
    L.muon_adamw_config_default.argtypes = [ctypes.POINTER(muon_adamw_config)]
    L.muon_adamw_config_default.restype = None
    L.muon_adamw_plan_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(muon_adamw_tensor),
                                         i64, ctypes.c_int]
    L.muon_adamw_plan_create.restype = ctypes.c_int
    L.muon_adamw_step.argtypes = [vp, ctypes.POINTER(vp), i64,
                                  ctypes.POINTER(muon_adamw_config), vp]
    L.muon_adamw_step.restype = ctypes.c_int
    L.muon_adamw_check.argtypes = [vp, ctypes.POINTER(vp), i64, ctypes.POINTER(muon_adamw_config)]
    L.muon_adamw_check.restype = ctypes.c_int
    L.muon_adamw_plan_table_size.argtypes = [vp]
    L.muon_adamw_plan_table_size.restype = sz
    L.muon_adamw_plan_upload.argtypes = [vp, vp, sz, vp]
    L.muon_adamw_plan_upload.restype = ctypes.c_int
    L.muon_adamw_plan_destroy.argtypes = [vp]
    L.muon_adamw_plan_destroy.restype = None
    L.muon_grad_plan_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(i64),
                                        ctypes.POINTER(ctypes.c_int), i64]
    L.muon_grad_plan_create.restype = ctypes.c_int
    L.muon_grad_plan_workspace_size.argtypes = [vp]
    L.muon_grad_plan_workspace_size.restype = sz
    L.muon_grad_norm.argtypes = [vp, ctypes.POINTER(vp), i64, ctypes.c_float, vp, vp, vp, sz, vp]
    L.muon_grad_norm.restype = ctypes.c_int
    L.muon_grad_scale.argtypes = [vp, ctypes.POINTER(vp), i64, vp, vp]
    L.muon_grad_scale.restype = ctypes.c_int
    L.muon_grad_plan_destroy.argtypes = [vp]
    L.muon_grad_plan_destroy.restype = None
    for size in (L.muon_mx_codes_size, L.muon_mx_scales_size):
        size.argtypes = [i64, i64]
        size.restype = sz
    L.muon_mx_quantize.argtypes = [ctypes.POINTER(muon_mx_source), i64, ctypes.c_int,
                                   ctypes.c_uint64, vp]
    L.muon_mx_quantize.restype = ctypes.c_int
    L.muon_mx_dequantize.argtypes = [vp, vp, i64, i64, vp, ctypes.c_int, vp]
    L.muon_mx_dequantize.restype = ctypes.c_int
    L.muon_mx_matmul_workspace_size.argtypes = [i64, i64, i64]
    L.muon_mx_matmul_workspace_size.restype = sz
    L.muon_mx_matmul.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, ctypes.c_int, vp, sz, vp]
    L.muon_mx_matmul.restype = ctypes.c_int
    L.muon_orthogonalize_workspace_size.argtypes = [i64, i64, i64, i64]
    L.muon_orthogonalize_workspace_size.restype = sz
    L.muon_orthogonalize_passes.argtypes = [ctypes.POINTER(muon_config)]
    L.muon_orthogonalize_passes.restype = ctypes.c_int
    L.muon_orthogonalize.argtypes = [ctypes.POINTER(muon_stack), ctypes.POINTER(muon_config), vp, sz, vp]
    L.muon_orthogonalize.restype = ctypes.c_int
    L.muon_status_string.argtypes = [ctypes.c_int]
    L.muon_status_string.restype = ctypes.c_char_p
    L.muon_last_error.argtypes = []
    L.muon_last_error.restype = ctypes.c_char_p
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().muon_status_string(int(status)).decode()


def raise_status(status: int) -> None:
    raise MuonError(status, muon_last_error())


def muon_last_error() -> str:
    return lib().muon_last_error().decode()


def _check(status: int) -> None:
    if status != MUON_OK:
        raise_status(status)


def muon_status_string(status: int) -> str:
    return status_string(status)


def muon_config_default() -> muon_config:
    cfg = muon_config()
    lib().muon_config_default(ctypes.byref(cfg))
    return cfg


def muon_plan_create(rows: Sequence[int], cols: Sequence[int], param_dtype: Sequence[int],
                     grad_dtype: Sequence[int], precision: int = MUON_NS_BF16) -> int:
    n = len(rows)
    if not (len(cols) == len(param_dtype) == len(grad_dtype) == n):
        raise ValueError("rows, cols, param_dtype and grad_dtype must have the same length")
    plan = ctypes.c_void_p()
    arr = lambda t, xs: (t * max(n, 1))(*xs)  # noqa: E731
    _check(lib().muon_plan_create(ctypes.byref(plan), arr(ctypes.c_int64, rows),
                                  arr(ctypes.c_int64, cols), arr(ctypes.c_int, param_dtype),
                                  arr(ctypes.c_int, grad_dtype), n, int(precision)))
    return plan.value


def muon_plan_workspace_size(plan: int) -> int:
    return int(lib().muon_plan_workspace_size(plan))


def muon_plan_destroy(plan: int) -> None:
    lib().muon_plan_destroy(plan)


def muon_step(plan: int, mats, n: int, cfg: muon_config, workspace: int, workspace_bytes: int,
              stream: int) -> None:
    """``mats``: a ctypes array of muon_matrix (or None when n == 0)."""
    _check(lib().muon_step(plan, mats, n, ctypes.byref(cfg), workspace, workspace_bytes, stream))


def muon_step_noalloc(plan: int, mats, n: int, cfg: muon_config, stream: int) -> None:
    """muon_step with the library's static device scratch instead of a workspace."""
    _check(lib().muon_step_noalloc(plan, mats, n, ctypes.byref(cfg), stream))


def muon_newton_schulz(plan: int, inputs: Sequence[int], outputs: Sequence[int],
                       cfg: muon_config, workspace: int, workspace_bytes: int,
                       stream: int) -> None:
    n = len(inputs)
    ins = (ctypes.c_void_p * max(n, 1))(*inputs)
    outs = (ctypes.c_void_p * max(n, 1))(*outputs)
    _check(lib().muon_newton_schulz(plan, ins, outs, n, ctypes.byref(cfg), workspace,
                                    workspace_bytes, stream))


def muon_plan_set_profiling(plan: int, enable: bool) -> None:
    _check(lib().muon_plan_set_profiling(plan, 1 if enable else 0))


def muon_plan_set_concurrency(plan: int, streams: int) -> None:
    _check(lib().muon_plan_set_concurrency(plan, int(streams)))


def muon_plan_set_fused(plan: int, enable: bool) -> None:
    _check(lib().muon_plan_set_fused(plan, 1 if enable else 0))


def muon_plan_read_profile(plan: int) -> dict:
    k = len(KERNEL_KINDS)
    ms = (ctypes.c_double * k)()
    n = (ctypes.c_int64 * k)()
    _check(lib().muon_plan_read_profile(plan, ms, n, k))
    return {name: (ms[i], n[i]) for i, name in enumerate(KERNEL_KINDS)}


def make_matrices(entries) -> ctypes.Array:
    """entries: iterable of (param_ptr, grad_ptr, momentum_ptr, out_ptr, rows, cols, pdt, gdt
    [, row_var_ptr])."""
    entries = list(entries)
    arr = (muon_matrix * max(len(entries), 1))()
    for i, e in enumerate(entries):
        arr[i] = muon_matrix(*e)
    return arr


def muon_adam_config_default() -> muon_adam_config:
    cfg = muon_adam_config()
    lib().muon_adam_config_default(ctypes.byref(cfg))
    return cfg


def muon_cautious_adam_step(tensors, n: int, cfg: muon_adam_config, stream: int) -> None:
    """``tensors``: a ctypes array of muon_adam_tensor (or None when n == 0)."""
    _check(lib().muon_cautious_adam_step(tensors, n, ctypes.byref(cfg), stream))


def make_adam_tensors(entries) -> ctypes.Array:
    """entries: iterable of (param, grad, exp_avg, exp_avg_sq, numel, pdt, gdt, wd_mul)."""
    entries = list(entries)
    arr = (muon_adam_tensor * max(len(entries), 1))()
    for i, e in enumerate(entries):
        arr[i] = muon_adam_tensor(*e)
    return arr


def muon_adamw_config_default() -> muon_adamw_config:
    cfg = muon_adamw_config()
    lib().muon_adamw_config_default(ctypes.byref(cfg))
    return cfg


def make_adamw_tensors(entries) -> ctypes.Array:
    """entries: iterable of (param, master, exp_avg, exp_avg_sq, exp_avg_scale,
    exp_avg_sq_scale, numel, pdt, gdt, wd_mul)."""
    entries = list(entries)
    arr = (muon_adamw_tensor * max(len(entries), 1))()
    for i, e in enumerate(entries):
        arr[i] = muon_adamw_tensor(*e)
    return arr


def pack_adamw_tensors(columns) -> ctypes.Array:
    """The same from whole columns of those fields (None: a NULL pointer)."""
    rows = list(zip(*columns))
    pack = struct.Struct("@6Pqiif0q").pack
    raw = b"".join(pack(*[x or 0 for x in r[:6]], *r[6:]) for r in rows)
    return (muon_adamw_tensor * max(len(rows), 1)).from_buffer_copy(
        raw or bytes(ctypes.sizeof(muon_adamw_tensor)))


def make_pointers(pointers: Sequence) -> ctypes.Array:
    return (ctypes.c_void_p * max(len(pointers), 1))(*pointers)


def muon_adamw_plan_create(tensors, n: int, state: int) -> int:
    """``tensors``: a ctypes array of muon_adamw_tensor (or None when n == 0)."""
    plan = ctypes.c_void_p()
    _check(lib().muon_adamw_plan_create(ctypes.byref(plan), tensors, n, int(state)))
    return plan.value


def muon_adamw_plan_table_size(plan: int) -> int:
    return int(lib().muon_adamw_plan_table_size(plan))


def muon_adamw_plan_upload(plan: int, table: int, table_bytes: int, stream: int) -> None:
    _check(lib().muon_adamw_plan_upload(plan, table, table_bytes, stream))


def muon_adamw_step(plan: int, grads, n: int, cfg: muon_adamw_config, stream: int) -> None:
    """``grads``: a ctypes array of pointers (make_pointers)."""
    _check(lib().muon_adamw_step(plan, grads, n, ctypes.byref(cfg), stream))


def muon_adamw_check(plan: int, grads, n: int, cfg: muon_adamw_config) -> None:
    _check(lib().muon_adamw_check(plan, grads, n, ctypes.byref(cfg)))


def muon_adamw_plan_destroy(plan: int) -> None:
    lib().muon_adamw_plan_destroy(plan)


def muon_grad_plan_create(numel: Sequence[int], dtype: Sequence[int]) -> int:
    n = len(numel)
    if len(dtype) != n:
        raise ValueError("numel and dtype must have the same length")
    plan = ctypes.c_void_p()
    _check(lib().muon_grad_plan_create(ctypes.byref(plan), (ctypes.c_int64 * max(n, 1))(*numel),
                                       (ctypes.c_int * max(n, 1))(*dtype), n))
    return plan.value


def muon_grad_plan_workspace_size(plan: int) -> int:
    return int(lib().muon_grad_plan_workspace_size(plan))


def muon_grad_norm(plan: int, grads, n: int, max_norm: float, out: int, norms, workspace: int,
                   workspace_bytes: int, stream: int) -> None:
    _check(lib().muon_grad_norm(plan, grads, n, max_norm, out, norms, workspace, workspace_bytes,
                                stream))


def muon_grad_scale(plan: int, grads, n: int, scale: int, stream: int) -> None:
    _check(lib().muon_grad_scale(plan, grads, n, scale, stream))


def muon_grad_plan_destroy(plan: int) -> None:
    lib().muon_grad_plan_destroy(plan)


def muon_mx_codes_size(rows: int, cols: int) -> int:
    return int(lib().muon_mx_codes_size(rows, cols))


def muon_mx_scales_size(rows: int, cols: int) -> int:
    return int(lib().muon_mx_scales_size(rows, cols))


def make_mx_sources(entries) -> ctypes.Array:
    """entries: iterable of (x, rows, cols, row_stride, dtype, codes, scales, codes_t, scales_t)."""
    entries = list(entries)
    arr = (muon_mx_source * max(len(entries), 1))()
    for i, e in enumerate(entries):
        arr[i] = muon_mx_source(*e)
    return arr


def muon_mx_quantize(sources, n: int, stochastic: int, seed: int, stream: int) -> None:
    """``sources``: a ctypes array of muon_mx_source (or None when n == 0)."""
    _check(lib().muon_mx_quantize(sources, n, int(stochastic), seed, stream))


def muon_mx_dequantize(codes: int, scales: int, rows: int, cols: int, out: int, dtype: int,
                       stream: int) -> None:
    _check(lib().muon_mx_dequantize(codes, scales, rows, cols, out, dtype, stream))


def muon_mx_matmul_workspace_size(m: int, n: int, k: int) -> int:
    return int(lib().muon_mx_matmul_workspace_size(m, n, k))


def muon_mx_matmul(a_codes: int, a_scales: int, b_codes: int, b_scales: int, m: int, n: int, k: int,
                   out: int, dtype: int, workspace, workspace_bytes: int, stream: int) -> None:
    _check(lib().muon_mx_matmul(a_codes, a_scales, b_codes, b_scales, m, n, k, out, dtype,
                                workspace, workspace_bytes, stream))


def muon_orthogonalize_workspace_size(outer: int, inner: int, rows: int, cols: int) -> int:
    return int(lib().muon_orthogonalize_workspace_size(outer, inner, rows, cols))


def muon_orthogonalize_passes(cfg: muon_config) -> int:
    passes = lib().muon_orthogonalize_passes(ctypes.byref(cfg))
    _check(min(passes, 0))
    return passes


def muon_orthogonalize(stack: muon_stack, cfg: muon_config, workspace, workspace_bytes: int,
                       stream: int) -> None:
    _check(lib().muon_orthogonalize(ctypes.byref(stack), ctypes.byref(cfg), workspace,
                                    workspace_bytes, stream))
