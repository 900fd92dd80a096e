"""Microscaled 4-bit values: quantisation, product, and a linear layer's three products over both,
PyTorch-facing wrappers of include/mx4.h.

A matrix is held in blocks of 32 values of a row: a code of 4 bits for each (a sign and one of 0,
1/2, 1, 3/2, 2, 3, 4, 6) and a power of two that the block shares. ``MX4Tensor`` is one held so,
``MX4Copies`` the held weights of a model, which ``Muon(mx4_copies=...)`` refreshes at the end of
every step. PyTorch supplies device memory and the current stream; the work runs in libmuon.so.

The pages' model pairs the optimizer with such products: a product with its two backward ones, held
operands in two layouts, and weights held anew after every step (there in 8 bits, the least that its
hardware multiplies).
"""
from __future__ import annotations

from typing import Dict, Iterable, Optional, Tuple

import torch

from . import _lib as L
from .adamw import _raw_stream
from .optim import dtype_code

_ROWS, _COLS, _BOTH = b"\1", b"\2", b"\3"


class MX4Tensor:
    """A matrix in microscaled 4-bit values, rows of its last dimension (leading dimensions, if
    any, are kept in ``shape``), outside of autograd: no derivative passes through it. ``data``: its
    codes and scales in the layout of include/mx4.h.

    ``MX4Tensor(codes, scales, cols)`` makes one from the usual layout: ``codes`` uint8, rows x at
    least ceil(cols / 2), the first of two codes in the low half; ``scales`` uint8 (or
    float8_e8m0fnu), rows x at least ceil(cols / 32). ``parts()`` is the way back."""

    __slots__ = ("data", "rows", "cols", "shape")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int):
        cols = int(cols)
        if scales.dtype == torch.float8_e8m0fnu:
            scales = scales.view(torch.uint8)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if codes.dim() != 2 or scales.dim() != 2 or codes.shape[0] != scales.shape[0]:
            raise ValueError("codes and scales must be 2-D, with equal rows")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        half, blocks = -(-cols // 2), -(-cols // 32)
        if cols < 0 or codes.shape[1] < half or scales.shape[1] < blocks:
            raise ValueError(f"{cols} columns need {half} bytes of codes and {blocks} of scales a row")
        rows = codes.shape[0]
        panels, steps = -(-rows // 16), -(-cols // 128)
        c = codes.new_zeros(panels * 16, steps * 64)
        c[:rows, :half] = codes[:, :half]
        if cols % 2:
            c[:rows, half - 1] &= 15
        s = scales.new_zeros(panels * 16, steps * 4)
        s[:rows, :blocks] = scales[:, :blocks]
        tiled = [t.view(panels, 16, steps, w).transpose(1, 2).reshape(-1) for t, w in ((c, 64), (s, 4))]
        self._set(torch.cat(tiled), rows, cols, (rows, cols))

    def _set(self, data, rows, cols, shape):
        self.data, self.rows, self.cols, self.shape = data, rows, cols, torch.Size(shape)

    @classmethod
    def _of(cls, data, rows, cols, shape) -> "MX4Tensor":
        t = object.__new__(cls)
        t.data, t.rows, t.cols, t.shape = data, rows, cols, shape
        return t

    @property
    def device(self) -> torch.device:
        return self.data.device

    def __repr__(self):
        return f"MX4Tensor(shape={tuple(self.shape)}, device={self.device})"

    def parts(self) -> Tuple[torch.Tensor, torch.Tensor]:
        """(codes, scales): uint8, rows x ceil(cols / 2) and rows x ceil(cols / 32)."""
        panels, steps = -(-self.rows // 16), -(-self.cols // 128)
        at = panels * steps * 1024
        codes = self.data[:at].view(panels, steps, 16, 64).transpose(1, 2).reshape(panels * 16, steps * 64)
        scales = self.data[at:].view(panels, steps, 16, 4).transpose(1, 2).reshape(panels * 16, steps * 4)
        return (codes[:self.rows, :-(-self.cols // 2)].contiguous(),
                scales[:self.rows, :-(-self.cols // 32)].contiguous())

    def dequantize(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """The values held, exactly, as bfloat16 or float32."""
        out = L.args().mx_dequantize(self.data, self.rows, self.cols, dtype_code(dtype))
        if type(out) is int:
            L.raise_status(out)
        return _shaped(out, self.shape)


def _shaped(out: torch.Tensor, shape) -> torch.Tensor:
    """out in another shape, and no view: one made under no_grad may not be changed with a graph later."""
    return out if len(shape) == 2 else torch.ops.aten._unsafe_view(out, shape)


def _quantize(tensors: tuple, results: bytes, stochastic: bool, seed: int):
    out = L.args().mx_quantize(tensors, results, stochastic, seed & (2 ** 64 - 1))
    if type(out) is int:
        L.raise_status(out)
    return out


def mx4_quantize(x: torch.Tensor, *, stochastic: bool = False, seed: int = 0) -> MX4Tensor:
    """x (bfloat16 or float32, rows of its last dimension, along which a product sums) in
    microscaled 4-bit values: to nearest, or stochastically with the random bits of ``seed``, which
    depend on it and on a value's place alone. x may have one stride between rows, or be the
    transpose of such a matrix."""
    rows, cols, data, _ = _quantize((x,), _ROWS, stochastic, seed)[0]
    return MX4Tensor._of(data, rows, cols, x.shape)


def mx4_quantize_both(x: torch.Tensor, *, stochastic: bool = False,
                      seed: int = 0) -> Tuple[MX4Tensor, MX4Tensor]:
    """(mx4_quantize(x), mx4_quantize(x^T)) in one pass over x, whose leading dimensions are one in
    the transpose."""
    rows, cols, data, turned = _quantize((x,), _BOTH, stochastic, seed)[0]
    return (MX4Tensor._of(data, rows, cols, x.shape),
            MX4Tensor._of(turned, cols, rows, torch.Size((cols, rows))))


def mx4_matmul(a: MX4Tensor, b: MX4Tensor, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """a b^T, along the last dimension of both: summed in float32 and rounded once to ``out_dtype``
    (bfloat16 or float32). The result has a's leading dimensions and b's rows."""
    if not isinstance(a, MX4Tensor) or not isinstance(b, MX4Tensor):
        raise TypeError("two MX4Tensors expected")
    if a.cols != b.cols:
        raise ValueError(f"last dimensions differ: {a.cols} and {b.cols}")
    out = L.args().mx_matmul(a.data, b.data, a.rows, b.rows, a.cols, dtype_code(out_dtype))
    if type(out) is int:
        L.raise_status(out)
    return _shaped(out, (*a.shape[:-1], b.rows))


def mx4_linear(x: torch.Tensor, weight: torch.Tensor,
               copies: Optional[Tuple[MX4Tensor, MX4Tensor]] = None, *, stochastic: bool = False,
               seed: int = 0) -> torch.Tensor:
    """x weight^T with all three products of the layer in microscaled 4-bit values: x (.., inputs)
    and weight (outputs, inputs), bfloat16 or float32. The result has x's dtype, gradients those of
    x and weight. Either may lie in any way; what ``mx4_quantize`` does not take is copied first. ``copies``: the weight and its transpose as held (``MX4Copies``), else the
    weight is quantised in this call. Values are rounded to nearest; ``stochastic``: but the incoming
    gradients stochastically, with the random bits of ``seed`` (give another for every step and layer; a
    captured pass repeats its own). As with any layer, let go of what an eager pass left of the graph of
    these leaves before a backward pass is captured. Differentiable once."""
    if not isinstance(x, torch.Tensor) or not isinstance(weight, torch.Tensor):
        raise TypeError("x and weight must be tensors")
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"x (.., inputs) and weight (outputs, inputs) expected, got {tuple(x.shape)} "
                         f"and {tuple(weight.shape)}")
    dtype_code(x.dtype), dtype_code(weight.dtype)
    if not x.is_cuda or weight.device != x.device:
        raise ValueError("x and weight must be on one CUDA device")
    if copies is not None:
        r, c = copies
        if (r.rows, r.cols) != tuple(weight.shape) or (c.cols, c.rows) != tuple(weight.shape):
            raise ValueError("copies of another shape than the weight's")
        if r.device != x.device or c.device != x.device:
            raise ValueError("copies on another device than x")
    rows, cols = (None, None) if copies is None else (copies[0].data, copies[1].data)
    seed = int(seed) & (2 ** 64 - 1)
    y = L.args().mx_linear(x, weight, rows, cols, bool(stochastic), seed - ((seed >> 63) << 64))
    if type(y) is int:
        L.raise_status(y)
    return y


class MX4Copies:
    """The held form of 2-D parameters and of their transposes, made here and again by
    ``refresh()``, one launch for up to 60 matrices of a dtype. ``copies[p]`` is the pair that
    ``mx4_linear`` takes. They follow what ``refresh`` saw: whoever changes a parameter otherwise than
    by ``Muon(mx4_copies=...)`` calls it. A backward pass over copies that were refreshed since its
    forward pass is refused by autograd."""

    def __init__(self, params: Iterable[torch.Tensor]):
        self._params = list(params)
        self._pairs: Dict[torch.Tensor, Tuple[MX4Tensor, MX4Tensor]] = {}
        for p in self._params:
            if not isinstance(p, torch.Tensor):
                raise TypeError("tensors expected")
            if p.dim() != 2 or not p.is_cuda or not p.is_contiguous():
                raise ValueError("contiguous 2-D CUDA parameters expected")
            if p.device != self._params[0].device:
                raise ValueError("all parameters must be on one device")
            if p in self._pairs:
                raise ValueError("a parameter stands in the list twice")
            dtype_code(p.dtype)
            sizes = [tuple(p.shape), tuple(p.shape)[::-1]]
            self._pairs[p] = tuple(
                MX4Tensor._of(torch.empty(L.muon_mx_codes_size(*s) // 16 * 17, dtype=torch.uint8,
                                          device=p.device), *s, torch.Size(s)) for s in sizes)
        self._at, self._sources = None, None
        self.refresh()

    def __len__(self):
        return len(self._params)

    def __getitem__(self, p: torch.Tensor) -> Tuple[MX4Tensor, MX4Tensor]:
        return self._pairs[p]

    def _entry(self, p):
        held = []
        for q in self._pairs[p]:
            at = q.data.data_ptr()
            held += [at, at + L.muon_mx_codes_size(q.rows, q.cols)] if at else [None, None]
        return (p.data_ptr(), *p.shape, p.shape[1], dtype_code(p.dtype), *held)

    @torch.no_grad()
    def refresh(self) -> None:
        """Quantises the parameters as they are now, on the current stream."""
        self._look()
        self._make()

    def _look(self):
        """Where the parameters are now: one may have been given other memory since (p.data = ...)."""
        now = [(p.data_ptr(), p.dtype, p.shape, p.is_contiguous()) for p in self._params]
        if now != self._at:
            for p in self._params:
                if tuple(p.shape) != (self._pairs[p][0].rows, self._pairs[p][0].cols) or \
                        not p.is_contiguous() or p.device != self._pairs[p][0].device:
                    raise ValueError("a parameter has another shape, layout or device than when its "
                                     "copies were made")
            self._sources = L.make_mx_sources(self._entry(p) for p in self._params)
            self._at = now

    def _make(self):
        if not self._params:
            return
        device = self._params[0].device
        with torch.cuda.device(device):
            L.muon_mx_quantize(self._sources, len(self._params), 0, 0, _raw_stream(device.index))
        for pair in self._pairs.values():
            torch.autograd.graph.increment_version([q.data for q in pair])
