"""AdamW over many tensors at once (fp32 or 8-bit states) and the gradient norm that clips it:
PyTorch-facing wrappers of include/adamw.h and include/grad_norm.h.

``AdamWPlan`` and ``GradNormPlan`` hold a plan of the library for a fixed list of tensors;
``AdamW`` is the ``torch.optim`` front end, ``clip_grad_norm_`` the in-place form for the other
optimizers. PyTorch supplies device memory and the current stream; every step runs in
libmuon.so.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import operator
from typing import Iterable, Optional, Sequence, Union

import torch

from . import _lib as L
from .optim import dtype_code

_NOTHING = contextlib.nullcontext()
_NONE = type(None)
_STATES = ("exp_avg", "exp_avg_sq", "master", "exp_avg_scale", "exp_avg_sq_scale")
_SCALE_AT = L.muon_adamw_config.grad_scale.offset
# the current stream's handle without a Stream object around it (2 us of a 10 us step)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or (
    torch.cuda.is_current_stream_capturing)


def make_adamw_config(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, step=1,
                      skip_nonfinite=False, stochastic=True, seed=0) -> L.muon_adamw_config:
    """A muon_adamw_config; ``step`` is the index t >= 1 of the step in the bias corrections.
    ``stochastic`` and ``seed``: how 8-bit states round the second moment."""
    cfg = L.muon_adamw_config_default()
    cfg.lr, cfg.beta1, cfg.beta2 = lr, betas[0], betas[1]
    cfg.eps, cfg.weight_decay, cfg.step = eps, weight_decay, int(step)
    cfg.skip_nonfinite, cfg.stochastic = int(bool(skip_nonfinite)), int(bool(stochastic))
    cfg.seed = int(seed) & (2 ** 64 - 1)
    return cfg


_MEAN_TOP, _ROOT_TOP = 240.0 * 2.0 ** 120, 240.0 * 2.0 ** 56   # the largest |m| and r held


def _hold(x: torch.Tensor, lost: torch.Tensor, floor: bool = False):
    """x (fp32, within the range held) as e4m3 codes, rounded to nearest, and the scales of its
    blocks; NaN where ``lost``. ``floor``: an x over zero does not become zero."""
    rows = x.new_zeros(-(-x.numel() // L.MUON_ADAMW_BLOCK), L.MUON_ADAMW_BLOCK)
    rows.view(-1)[:x.numel()] = x.flatten()
    top = rows.abs().nan_to_num(0.0).amax(1)
    # top = 2^(E - 127) f has the scale byte E - 8, or E - 7 where f is over 1 + 0x629146 / 2^23
    byte = (((top.view(torch.int32) + (0x7fffff - 0x629146)) >> 23) - 8).clamp_min(0).int()
    y = (rows * ((254 - byte) << 23).view(torch.float32)[:, None]).clamp(-448.0, 448.0)
    if floor:
        y = torch.where(rows > 0, y.clamp_min(2.0 ** -9), y)
    y = y.view(-1)[:x.numel()].view(x.shape).masked_fill(lost, math.nan)
    return y.to(torch.float8_e4m3fn), byte.to(torch.uint8).view(torch.float8_e8m0fnu)


def _one_device(tensors: Sequence[torch.Tensor]) -> torch.device:
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("CUDA tensors expected")
        if t.device != tensors[0].device:
            raise ValueError("all tensors must be on one device")
    if tensors:
        return tensors[0].device
    return torch.device("cuda", torch.cuda.current_device() if torch.cuda.is_available() else 0)


class _TensorList:
    """The device and gradient layout shared by the two plans."""

    def _set_list(self, device, numels, dtypes):
        n = len(numels)
        self.device = device
        self._numels = (ctypes.c_int64 * n)(*numels)
        self._dtypes = (ctypes.c_int32 * n)(*[dtype_code(d) for d in dtypes])

    def _list(self, grads: Sequence[Optional[torch.Tensor]]):
        if not isinstance(grads, (list, tuple)):
            grads = list(grads)
        if len(grads) != len(self._numels):
            raise ValueError(f"expected {len(self._numels)} gradients, got {len(grads)}")
        return grads

    def _refuse(self, grads, code: int):
        """Raises for what a native call returned: a gradient's index, or a status below 0."""
        if code < 0:
            L.raise_status(code)
        g = grads[code]
        if not isinstance(g, torch.Tensor):
            raise TypeError(f"gradient {code}: a tensor or None expected")
        if g.numel() != self._numels[code] or not g.is_contiguous() or g.device != self.device:
            raise ValueError(f"gradient {code}: a contiguous tensor of {self._numels[code]} "
                             f"elements on {self.device} expected")
        if dtype_code(g.dtype) == self._dtypes[code]:
            raise ValueError(f"gradient {code}: a tensor whose memory holds its values expected")
        raise TypeError(f"gradient {code}: a dtype other than the plan's ({g.dtype})")

    def fits(self, grads: Sequence[torch.Tensor]) -> bool:
        """Whether the gradients have the plan's sizes, dtypes and device, and are contiguous."""
        return (len(grads) == len(self._numels) and
                not isinstance(L.tensor_addresses(grads, self._numels, self._dtypes,
                                                  self.device.index), int))

    def _on(self, stream):
        """A context with the plan's device as the current one and ``stream`` (or the current
        stream) as its current stream."""
        if stream is not None:
            if stream.device != self.device:
                raise ValueError(f"the stream must be one of {self.device}")
            return torch.cuda.stream(stream)
        if torch.cuda.current_device() != self.device.index:
            return torch.cuda.device(self.device)
        return _NOTHING

    def _stream(self):
        return _raw_stream(self.device.index)


class AdamWPlan(_TensorList):
    """A plan of the library for a fixed list of parameters and their states, which it holds.

    ``exp_avgs`` and ``exp_avg_sqs``: float32, or all float8_e4m3fn (the 8-bit states, the
    second one holding sqrt(v)) with ``exp_avg_scales`` and ``exp_avg_sq_scales``, one
    float8_e8m0fnu per 256 elements of a tensor. ``grad_dtypes``: of the gradients that steps
    will receive. ``masters``: per parameter None or, for a bfloat16 one, its float32 master
    copy. ``wd_muls``: per parameter the multiplier of the weight decay (default 1). All
    contiguous and, scales apart, starting at multiples of 16 bytes; all states and scales zero
    before step 1. Making a plan waits once for the current stream, which fills its table."""

    def __init__(self, params: Sequence[torch.Tensor], exp_avgs: Sequence[torch.Tensor],
                 exp_avg_sqs: Sequence[torch.Tensor], grad_dtypes: Sequence[torch.dtype],
                 masters: Optional[Sequence[Optional[torch.Tensor]]] = None,
                 exp_avg_scales: Optional[Sequence[torch.Tensor]] = None,
                 exp_avg_sq_scales: Optional[Sequence[torch.Tensor]] = None,
                 wd_muls: Optional[Sequence[float]] = None):
        self.handle = None
        n = len(params)
        masters = [None] * n if masters is None else list(masters)
        wd_muls = [1.0] * n if wd_muls is None else [float(w) for w in wd_muls]
        if (exp_avg_scales is None) != (exp_avg_sq_scales is None):
            raise ValueError("give both scales or neither")
        small = exp_avg_scales is not None
        scales_m = list(exp_avg_scales) if small else [None] * n
        scales_r = list(exp_avg_sq_scales) if small else [None] * n
        lists = (exp_avgs, exp_avg_sqs, grad_dtypes, masters, scales_m, scales_r, wd_muls)
        if any(len(x) != n for x in lists):
            raise ValueError("one state, gradient dtype, master, scale and wd_mul per parameter")
        tensors = (params, masters, exp_avgs, exp_avg_sqs, scales_m, scales_r)
        grad_codes = [dtype_code(d) for d in grad_dtypes]
        codes = [dtype_code(p.dtype) for p in params]
        self._set_list(params[0].device if n else _one_device(()), [p.numel() for p in params],
                       grad_dtypes)
        blocks = [-(-k // L.MUON_ADAMW_BLOCK) for k in self._numels] if small else [0] * n
        ints = lambda xs: (ctypes.c_int32 * n)(*xs)  # noqa: E731
        sizes = [self._numels] * 4 + [(ctypes.c_int64 * n)(*blocks)] * 2
        state = ints([2 if small else 1] * n)
        dtypes = [ints(codes), ints([1] * n), state, state] + [ints([3] * n)] * 2
        index = self.device.index if self.device.type == "cuda" else -1
        at = [L.tensor_addresses(*x, index) for x in zip(tensors, sizes, dtypes)]
        if any(isinstance(x, int) for x in at):
            self._refuse_tensors(*tensors, torch.float8_e4m3fn if small else torch.float32)
        held = [t for ts in tensors for t in ts if t is not None]
        self.state_bits = 8 if small else 32
        packed = L.pack_adamw_tensors((*at, self._numels, codes, grad_codes, wd_muls))
        self.handle = L.muon_adamw_plan_create(packed if n else None, n,
                                               L.MUON_ADAMW_8BIT if small else L.MUON_ADAMW_F32)
        self._step = L.address_of(L.lib().muon_adamw_step)
        self._check = L.address_of(L.lib().muon_adamw_check)
        self._held = held
        self._table = self._made_on = None
        self.captured = False            # whether a graph may read the table
        size = L.muon_adamw_plan_table_size(self.handle)
        if size:
            with self._on(None):
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("create the plan before the capture")
                self._table = torch.empty(size, dtype=torch.uint8, device=self.device)
                self._made_on = self._stream()
                L.muon_adamw_plan_upload(self.handle, self._table.data_ptr(), size, self._made_on)
                torch.cuda.current_stream(self.device).synchronize()   # steps on any stream

    @staticmethod
    def _refuse_tensors(params, masters, exp_avgs, exp_avg_sqs, scales_m, scales_r, state_dtype):
        """Raises for the tensor that does not fit."""
        every = []
        for i, (p, w, m, v, ms, vs) in enumerate(zip(params, masters, exp_avgs, exp_avg_sqs,
                                                     scales_m, scales_r)):
            mine = [t for t in (p, w, m, v, ms, vs) if t is not None]
            if not all(isinstance(t, torch.Tensor) for t in mine):
                raise TypeError(f"parameter {i}: tensors expected")
            for t in (p, w, m, v):
                if t is not None and t.numel() != p.numel():
                    raise ValueError(f"parameter {i}: tensors of {p.numel()} elements expected")
            if any(not t.is_contiguous() for t in mine):
                raise ValueError(f"parameter {i}: contiguous tensors expected")
            if any(t is not None and t.dtype != state_dtype for t in (m, v)):
                raise TypeError(f"parameter {i}: states must be {state_dtype}: float8_e4m3fn beside "
                                "scales, float32 without")
            if w is not None and w.dtype != torch.float32:
                raise TypeError(f"parameter {i}: the master copy must be float32")
            for t in (ms, vs):
                if t is not None and t.dtype != torch.float8_e8m0fnu:
                    raise TypeError(f"parameter {i}: scales must be float8_e8m0fnu")
                if t is not None and t.numel() != -(-p.numel() // L.MUON_ADAMW_BLOCK):
                    raise ValueError(f"parameter {i}: one scale per {L.MUON_ADAMW_BLOCK} elements")
            every += mine
        _one_device(every)
        raise ValueError("a tensor that a plan cannot hold")

    def step(self, grads: Sequence[Optional[torch.Tensor]], cfg: L.muon_adamw_config,
             grad_scale: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> None:
        """One step. A gradient may be None: its parameter is left out. ``grad_scale``: one
        float32 on the device that every gradient is multiplied by (``GradNormPlan.norm``'s)."""
        grads = self._list(grads)
        with self._on(stream):
            on = self._stream()
            if on != self._made_on and self._table is not None:
                self._table.record_stream(torch.cuda.current_stream(self.device))
            self.captured = self.captured or _capturing()
            code = L.args().adamw_step(self._step, self.handle or 0, grads, self._numels, self._dtypes,
                                       self.device.index, cfg, grad_scale, _SCALE_AT, on)
        if code is not None:
            self._refuse(grads, code)

    def check(self, grads: Sequence[Optional[torch.Tensor]], cfg: L.muon_adamw_config,
              grad_scale: Optional[torch.Tensor] = None) -> None:
        """Raises what ``step`` would raise for these arguments; nothing is stepped."""
        grads = self._list(grads)
        code = L.args().adamw_check(self._check, self.handle or 0, grads, self._numels, self._dtypes,
                                    self.device.index, cfg, grad_scale, _SCALE_AT)
        if code is not None:
            self._refuse(grads, code)

    def close(self):
        if getattr(self, "handle", None):
            L.muon_adamw_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class GradNormPlan(_TensorList):
    """A plan of the library for gradients like those given (their sizes, dtypes and device;
    the tensors themselves are not kept)."""

    def __init__(self, grads: Sequence[torch.Tensor]):
        self.handle = None
        grads = list(grads)
        self._set_list(_one_device(grads), [g.numel() for g in grads], [g.dtype for g in grads])
        self.handle = L.muon_grad_plan_create(list(self._numels), list(self._dtypes))
        self.ws_bytes = L.muon_grad_plan_workspace_size(self.handle)
        self._norm = L.address_of(L.lib().muon_grad_norm)

    def norm(self, grads: Sequence[Optional[torch.Tensor]], max_norm: float = math.inf,
             per_tensor: bool = False, stream: Optional[torch.cuda.Stream] = None):
        """(norm, scale), or with ``per_tensor`` (norm, scale, norms): float32 on the device,
        new tensors each call. scale = min(1, max_norm / norm), NaN for a norm that is not
        finite. A gradient that is None counts as zero. The workspace belongs to the call."""
        grads = self._list(grads)
        with self._on(stream):
            out = L.args().grad_norm(self._norm, self.handle or 0, grads, self._numels, self._dtypes,
                                     self.device.index, max_norm, per_tensor, self.ws_bytes,
                                     self._stream())
        if isinstance(out, int):
            self._refuse(grads, out)
        return out

    def scale_(self, grads: Sequence[Optional[torch.Tensor]], scale: torch.Tensor,
               stream: Optional[torch.cuda.Stream] = None) -> None:
        """Multiplies every gradient by ``scale`` (one float32 on the device) in place; where it
        is 1 nothing is read or written."""
        grads = self._list(grads)
        if scale.numel() != 1 or scale.dtype != torch.float32 or scale.device != self.device:
            raise ValueError(f"scale must be one float32 on {self.device}")
        ptrs = L.tensor_addresses(grads, self._numels, self._dtypes, self.device.index)
        if isinstance(ptrs, int):
            self._refuse(grads, ptrs)
        with self._on(stream):
            L.muon_grad_scale(self.handle, ptrs, len(ptrs), scale.data_ptr(), self._stream())

    def close(self):
        if getattr(self, "handle", None):
            L.muon_grad_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def grad_norm(grads: Iterable[torch.Tensor], max_norm: float = math.inf):
    """(norm, scale) of a list of CUDA gradients (bfloat16 or float32, contiguous, starting at
    multiples of 16 bytes)."""
    grads = list(grads)
    return GradNormPlan(grads).norm(grads, max_norm)


def clip_grad_norm_(parameters: Union[torch.Tensor, Iterable[torch.Tensor]],
                    max_norm: float) -> torch.Tensor:
    """Scales the gradients of ``parameters`` in place to a global 2-norm of at most
    ``max_norm`` and returns their norm before it (a float32 on the device; nothing
    synchronises). If the norm is not finite, every gradient becomes NaN. Gradients are
    contiguous, on one device, start at multiples of 16 bytes and do not overlap (a view into a
    bucket of odd-sized tensors may start elsewhere: MuonError, and no gradient changes)."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    plan = GradNormPlan(grads)
    norm, scale = plan.norm(grads, max_norm)
    plan.scale_(grads, scale)
    return norm


class AdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay for any parameters (bfloat16 or float32, contiguous,
    one device per group), one pass over all tensors of a group.

    ``state_bits``: 32, or 8 for e4m3 moments with a power-of-two scale per 256 elements
    (``stochastic``, ``seed``: the rounding of the second one). ``master_weights``: bfloat16
    parameters get a float32 master copy (``refresh_masters`` rereads it after the parameters
    were set from outside). ``wd_mul``: multiplier of ``weight_decay``. These and the
    hyper-parameters may differ by group. ``max_grad_norm``: clips the gradients' global norm
    over all groups, inside the step (the gradients themselves stay as they are);
    ``skip_nonfinite`` leaves a step out whose norm is not finite (its index still counts).
    ``last_grad_norm`` is the norm of the last step that had either, on the device. A step under
    graph capture replays with the index, and so the bias corrections and the random bits, that
    it was captured with.

    A parameter without a gradient is left out of a step. A step waits for the current stream only
    where it meets a parameter's gradient for the first time, or after parameters, states,
    gradients' dtypes or ``wd_mul`` were exchanged from outside (a new plan's table is filled then);
    such a step cannot be captured. Parameters, states and gradients start at multiples of 16
    bytes."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, wd_mul: float = 1.0, state_bits: int = 32,
                 master_weights: bool = False, stochastic: bool = True, seed: int = 0,
                 max_grad_norm: Optional[float] = None, skip_nonfinite: bool = False):
        defaults = dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay,
                        wd_mul=wd_mul, state_bits=state_bits, master_weights=master_weights,
                        stochastic=stochastic, seed=seed)
        if max_grad_norm is not None and not max_grad_norm >= 0.0:
            raise ValueError(f"max_grad_norm must be >= 0, not {max_grad_norm}")
        self._plans = {}
        self._every = []                 # the parameters' states that the plans were checked with
        self._captured = []              # plans no longer used here that a graph may replay
        self.max_grad_norm = max_grad_norm
        self.skip_nonfinite = skip_nonfinite
        self.last_grad_norm = None
        super().__init__(params, defaults)

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        try:
            self._check_options(self.param_groups[-1])
        except Exception:
            self.param_groups.pop()
            raise

    @staticmethod
    def _check_options(group):
        """What no step would take, as torch.optim.AdamW has it, is refused here already. (Steps
        take fp32 options: a beta that rounds to 1 is one.)"""
        fp32 = lambda x: ctypes.c_float(float(x)).value  # noqa: E731
        if group["state_bits"] not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        for k in ("lr", "eps", "weight_decay"):
            if not 0.0 <= fp32(group[k]) < math.inf:
                raise ValueError(f"{k} must be finite and >= 0, not {group[k]}")
        if len(group["betas"]) != 2 or not all(0.0 <= fp32(b) < 1.0 for b in group["betas"]):
            raise ValueError(f"betas must be two numbers in [0, 1), not {group['betas']}")
        wd_mul = fp32(group["wd_mul"])
        if not math.isfinite(wd_mul) or not math.isfinite(fp32(wd_mul * fp32(group["weight_decay"]))):
            raise ValueError(f"wd_mul and wd_mul * weight_decay must be finite, not {group['wd_mul']} "
                             f"and {group['weight_decay']}")

    def __getstate__(self):
        state = super().__getstate__()
        state.update(max_grad_norm=self.max_grad_norm, skip_nonfinite=self.skip_nonfinite)
        return state

    def __setstate__(self, state):
        super().__setstate__(state)                  # load_state_dict calls this as well
        self.__dict__.setdefault("_plans", {})
        self.__dict__.setdefault("_captured", [])
        self._every = []
        for gi in list(self._plans):
            self._drop_plan(gi)
        self.last_grad_norm = None

    def load_state_dict(self, state_dict):
        """As the base class's, except that states keep the dtypes they were saved with. One of
        ``torch.optim.AdamW`` will do: its moments, in whatever dtype, become float32, or where the
        group has ``state_bits`` 8 the nearest 8-bit states, and where the group has
        ``master_weights`` the parameters' present values become the master copies; options that
        torch's does not have stay as each group has them. Options of torch's that would step
        otherwise (``amsgrad``, ``maximize``, the coupled decay of Adam) are refused."""
        for group in state_dict["param_groups"]:
            for k in ("amsgrad", "maximize"):
                if group.get(k):
                    raise ValueError(f"AdamW has no {k}")
            if group.get("decoupled_weight_decay") is False and group.get("weight_decay"):
                raise ValueError("AdamW's weight decay is decoupled")
        own = [{k: group.get(k, v) for k, v in self.defaults.items()}
               for group in self.param_groups]
        super().load_state_dict(state_dict)
        for group, options in zip(self.param_groups, own):
            for k, v in options.items():
                group.setdefault(k, v)
        ids = [i for g in state_dict["param_groups"] for i in g["params"]]
        ps = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(ids, ps):
            for k, v in state_dict["state"].get(i, {}).items():
                if k == "step":
                    self.state[p][k] = int(v)
                elif isinstance(v, torch.Tensor):
                    self.state[p][k] = v.detach().clone().to(p.device)
        for group in self.param_groups:
            for p in group["params"]:
                if p in self.state:
                    self._complete_state(p, self.state[p], group)

    @staticmethod
    def _complete_state(p, st, group):
        """Brings a loaded state to the form that the group's steps take."""
        if "exp_avg" not in st or "exp_avg_sq" not in st:          # another optimizer's
            return
        if "exp_avg_scale" not in st:
            m, v = (st[k].float().contiguous() for k in ("exp_avg", "exp_avg_sq"))
            if group["state_bits"] == 8:
                m, st["exp_avg_scale"] = _hold(m.clamp(-_MEAN_TOP, _MEAN_TOP), m.isinf())
                v, st["exp_avg_sq_scale"] = _hold(v.sqrt().clamp(max=_ROOT_TOP), v < 0, floor=True)
            st["exp_avg"], st["exp_avg_sq"] = m, v
        if "master" not in st and group["master_weights"] and p.dtype == torch.bfloat16:
            st["master"] = p.detach().float()

    def _drop_plan(self, gi):
        """Forgets a group's plan, unless a graph was captured with it: its table and the states
        that it was made for then stay allocated as long as the optimizer."""
        cached = self._plans.pop(gi, None)
        if gi != "norm" and cached is not None and cached[0].captured:
            self._captured.append(cached[0])

    def _init_state(self, p, group):
        """Makes p's state, or where memory runs out none of it."""
        st = {"step": 0}
        zeros = lambda shape, dt: torch.zeros(  # noqa: E731
            shape, dtype=torch.uint8 if dt.itemsize == 1 else dt, device=p.device).view(dt)
        if group["state_bits"] == 8:
            blocks = -(-p.numel() // L.MUON_ADAMW_BLOCK)
            for k in ("exp_avg", "exp_avg_sq"):
                st[k] = zeros(p.shape, torch.float8_e4m3fn)
                st[k + "_scale"] = zeros((blocks,), torch.float8_e8m0fnu)
        else:
            for k in ("exp_avg", "exp_avg_sq"):
                st[k] = zeros(p.shape, torch.float32)
        if group["master_weights"] and p.dtype == torch.bfloat16:
            st["master"] = p.detach().float()
        self.state[p].update(st)

    @torch.no_grad()
    def refresh_masters(self):
        """Sets the master copies to the parameters' present values."""
        for p, st in self.state.items():
            if "master" in st:
                st["master"].copy_(p)

    def _follow_states(self):
        """Drops the plans of groups whose states are other dicts by now. Looking a parameter up
        takes 0.2 us, so that is done only where the dicts of all parameters have changed."""
        every = self.state.values()
        if len(every) == len(self._every) and all(map(operator.is_, every, self._every)):
            return
        for gi, cached in list(self._plans.items()):
            if gi != "norm" and not all(self.state.get(p) is st
                                        for p, st in zip(cached[1], cached[3])):
                self._drop_plan(gi)
        self._every = list(self.state.values())

    @staticmethod
    def _in_order(of, ps, grads):
        """The gradients of the parameters ``of``, a part of ``ps``; None if another one has any."""
        if len(of) == len(ps) and all(map(operator.is_, of, ps)):
            return grads
        mine = []
        for p, g in zip(ps, grads):
            if len(mine) < len(of) and of[len(mine)] is p:
                mine.append(g)
            elif g is not None:
                return None
        return mine if len(mine) == len(of) else None

    def _plan(self, gi, group, grads):
        """The group's plan, the states of its parameters and their gradients. A plan is kept while
        its parameters, their states, both's addresses, the gradients' layout and the decay's
        multiplier stay; gradients may come and go. (Eager steps that leave parameters out go on
        with another one than a graph's.)"""
        ps = group["params"]
        cached = self._plans.get(gi)
        if cached is not None:
            plan, of, wd_mul, states, numels, pdt, at, states_at = cached
            mine = self._in_order(of, ps, grads)
            if (mine is not None and wd_mul == group["wd_mul"]
                    and L.args().entries_at(states, _STATES, states_at) and plan.fits(mine)
                    and not (plan.captured and any(g is None for g in mine) and not _capturing())):
                now = L.tensor_addresses(of, numels, pdt, plan.device.index)
                if not isinstance(now, int) and bytes(now) == at:
                    return plan, states, mine
        live = [(p, g) for p, g in zip(ps, grads) if g is not None]
        device = live[0][0].device
        if device.type == "cuda":
            with torch.cuda.device(device):
                if torch.cuda.is_current_stream_capturing():   # before a state is made in the graph
                    raise RuntimeError("AdamW: take a step with these parameters and gradients "
                                       "before the capture")
        for p, g in live:
            if not p.is_contiguous() or not g.is_contiguous():
                raise ValueError("AdamW needs contiguous parameters and gradients")
            if "step" not in self.state[p]:
                self._init_state(p, group)
        small = "exp_avg_scale" in self.state[live[0][0]]
        absent = self._unmoved(cached, device, small)
        try:
            return self._new_plan(gi, group, grads, absent, small)
        except L.MuonError:
            if not absent:
                raise
        return self._new_plan(gi, group, grads, {}, small)     # one lies where a live one is now

    def _new_plan(self, gi, group, grads, absent, small):
        """A plan of the parameters with gradients and of ``absent``: {id: gradient's dtype}."""
        of, mine, grad_dtypes = [], [], []
        for p, g in zip(group["params"], grads):
            if g is not None or id(p) in absent:
                of.append(p)
                mine.append(g)
                grad_dtypes.append(absent[id(p)] if g is None else g.dtype)
        states = [self.state[p] for p in of]
        if any(("exp_avg_scale" in st) != small for st in states):
            raise ValueError("a group's states must all have the same state_bits")
        plan = AdamWPlan([p.detach() for p in of], [s["exp_avg"] for s in states],
                         [s["exp_avg_sq"] for s in states], grad_dtypes,
                         [s.get("master") for s in states],
                         [s["exp_avg_scale"] for s in states] if small else None,
                         [s["exp_avg_sq_scale"] for s in states] if small else None,
                         [group["wd_mul"]] * len(of))
        self._drop_plan(gi)
        n = len(of)
        numels = (ctypes.c_int64 * n)(*[p.numel() for p in of])
        pdt = (ctypes.c_int32 * n)(*[dtype_code(p.dtype) for p in of])
        at = bytes((ctypes.c_void_p * n)(*[p.data_ptr() for p in of]))
        states_at = (ctypes.c_uint64 * (n * len(_STATES)))(
            *[st[k].data_ptr() if k in st else 0 for st in states for k in _STATES])
        self._plans[gi] = (plan, of, group["wd_mul"], states, numels, pdt, at, states_at)
        return plan, states, mine

    def _unmoved(self, cached, device, small):
        """Those parameters of a plan that are, with their states, where the plan has them, by id:
        the next plan holds them without a gradient too, so that sets which alternate share one."""
        if cached is None or cached[0].device != device:
            return {}
        plan, of, _, states, numels, pdt, at, states_at = cached
        dtypes, k, found = (torch.bfloat16, torch.float32), len(_STATES), {}
        for i, (p, st) in enumerate(zip(of, states)):
            now = L.tensor_addresses([p], (ctypes.c_int64 * 1)(numels[i]),
                                     (ctypes.c_int32 * 1)(pdt[i]), device.index)
            if (not isinstance(now, int) and bytes(now) == at[8 * i:8 * i + 8]
                    and self.state.get(p) is st and ("exp_avg_scale" in st) == small
                    and L.args().entries_at([st], _STATES, (ctypes.c_uint64 * k)(
                        *states_at[k * i:k * i + k]))):
                found[id(p)] = dtypes[plan._dtypes[i]]
        return found

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        self._follow_states()
        todo = []
        for gi, group in enumerate(self.param_groups):
            grads = [p.grad for p in group["params"]]
            absent = list(map(type, grads)).count(_NONE)
            if absent < len(grads):
                todo.append((group, *self._plan(gi, group, grads), absent > 0))
        scale = None
        if (self.max_grad_norm is not None or self.skip_nonfinite) and todo:
            every = [g for *_, grads, absent in todo
                     for g in (filter(torch.is_tensor, grads) if absent else grads)]
            plan = self._plans.get("norm")
            if plan is None or not plan.fits(every):
                plan = self._plans["norm"] = GradNormPlan(every)
            self.last_grad_norm, scale = plan.norm(
                every, math.inf if self.max_grad_norm is None else self.max_grad_norm)
        calls = []                       # (plan, gradients, configuration, states, their index)
        for group, plan, states, grads, absent in todo:
            at = ([0 if g is None else st["step"] + 1 for st, g in zip(states, grads)] if absent
                  else [st["step"] + 1 for st in states])
            ts = set(at) - {0}
            for t in sorted(ts):
                cfg = make_adamw_config(group["lr"], group["betas"], group["eps"],
                                        group["weight_decay"], t,
                                        self.skip_nonfinite,
                                        group["stochastic"], group["seed"])
                if len(ts) > 1:
                    mine = [g if k == t else None for g, k in zip(grads, at)]
                else:
                    mine = grads
                if len(ts) > 1 or absent:
                    states_t = [st for st, k in zip(states, at) if k == t]
                else:
                    states_t = states
                calls.append((plan, mine, cfg, states_t, t))
        if len(calls) > 1:               # none is made where a later one would be refused
            for plan, grads, cfg, *_ in calls:
                plan.check(grads, cfg, scale)
        for plan, grads, cfg, states, t in calls:
            plan.step(grads, cfg, scale)
            for st in states:
                st["step"] = t
        return loss
