"""Rows between two routings: the norm of the residual plus a token's expert rows, the gated
activation between the experts' products, their gradients, and rows in 8 bits (see
include/moe_route_sort.h).

``moe_*`` functions have the names of their C entry points and fill caller-owned buffers;
``fp8_quantize``, ``rms_norm``, ``rms_norm_backward``, ``swiglu`` and ``swiglu_backward`` allocate
what is not given.
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import load
from .marshal import DTYPE_CODE, Entry, cuda_device, made, need, rows_of

_quantize = Entry("moe_fp8_quantize")
_norm = Entry("moe_rms_norm")
_norm_backward = Entry("moe_rms_norm_backward")
_gated = Entry("moe_swiglu")
_gated_backward = Entry("moe_swiglu_backward")

FP8 = torch.float8_e4m3fn
_HALF = {torch.bfloat16: 0, torch.float16: 1}


def moe_rms_norm_backward_workspace_bytes(cols: int) -> int:
    return int(load().moe_rms_norm_backward_workspace_bytes(cols))


class Fp8Rows:
    """Rows in 8 bits: ``codes`` [..., cols] float8_e4m3fn and ``scales`` [...] float32, on one
    CUDA device; a value is code * scale.  Weights of E experts are [E, outs, cols].  The two
    tensors are checked here, once, and cannot be exchanged afterwards."""

    __slots__ = ("_codes", "_scales", "lead", "cols", "device")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        self.device = cuda_device(codes, "codes")
        self._codes, self._scales = codes, scales
        self.lead = tuple(codes.shape[:-1])
        self.cols = codes.shape[-1]
        if tuple(scales.shape) != self.lead:
            raise ValueError(f"scales must be {self.lead} for codes {tuple(codes.shape)}, got "
                             f"{tuple(scales.shape)}")
        need(codes, FP8, 0, self.device, "codes")
        need(scales, torch.float32, 0, self.device, "scales")

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    tensors = property(lambda self: (self._codes, self._scales))

    @classmethod
    def allocate(cls, rows, cols: int, device="cuda") -> "Fp8Rows":
        """Room for ``rows`` (a number, or a tuple such as (E, outs)) of ``cols`` elements."""
        lead = tuple(rows) if isinstance(rows, (tuple, list)) else (rows,)
        return cls(torch.empty(*lead, cols, dtype=FP8, device=device),
                   torch.empty(lead, dtype=torch.float32, device=device))


def _half(t: torch.Tensor, name: str) -> int:
    code = _HALF.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return code


def _optional(t, dtype, numel, dev, name) -> int:
    return 0 if t is None else need(t, dtype, numel, dev, name)


# ------------------------------------------------------------------------- rows in 8 bits
def moe_fp8_quantize(x, codes, scales, stream=None) -> None:
    """Rows of ``x`` (a matrix with dense rows: bfloat16, float16 or float32) into codes and
    scales."""
    dev = cuda_device(x, "x")
    if x.dtype not in DTYPE_CODE:
        raise ValueError(f"x must be bfloat16, float16 or float32, got {x.dtype}")
    rows, cols, stride = rows_of(x, "x")
    _quantize(dev, stream, x.data_ptr(), DTYPE_CODE[x.dtype], rows, cols, stride,
              need(codes, FP8, rows * cols, dev, "codes"),
              need(scales, torch.float32, rows, dev, "scales"))


def fp8_quantize(x, out: Optional[Fp8Rows] = None, stream=None) -> Fp8Rows:
    """Rows of ``x`` ([..., cols]) in 8 bits; allocates the result unless ``out`` is given."""
    dev = cuda_device(x, "x")
    shape = x.shape
    if x.dim() == 0:
        raise ValueError("x must have rows")
    if out is None:
        out = made(dev, stream, lambda: Fp8Rows.allocate(shape[:-1], shape[-1], device=x.device))
    elif out.lead != shape[:-1] or out.cols != shape[-1] or out.device != dev:
        raise ValueError(f"out holds rows of shape {tuple(out.codes.shape)} on cuda:{out.device}, "
                         f"x is {tuple(shape)} on {x.device}")
    if len(shape) != 2:
        given = x
        x = made(dev, stream, lambda: given.reshape(-1, shape[-1]))  # a copy, if not a view
    moe_fp8_quantize(x, out._codes, out._scales, stream)
    return out


# -------------------------------------------------------------------------------- the norm
class NormBuffers:
    """Outputs of the norm for one (T, cols): ``y`` and ``sum`` [T, cols] of the rows' type,
    ``rows8`` (Fp8Rows) and ``rstd`` [T] float32; what was not asked for is None.  The buffers are
    the container's own and cannot be exchanged."""

    __slots__ = ("_y", "_sum", "_rows8", "_rstd", "_shape", "_at")

    def __init__(self, T: int, cols: int, dtype, device, y: bool, sum: bool, fp8: bool, rstd: bool):
        if dtype not in _HALF:
            raise ValueError(f"rows must be bfloat16 or float16, got {dtype}")
        if not (y or sum or fp8 or rstd):
            raise ValueError("a norm needs an output: y, sum, fp8 or rstd")

        def half(wanted):
            return torch.empty(T, cols, dtype=dtype, device=device) if wanted else None

        self._y, self._sum = half(y), half(sum)
        self._rows8 = Fp8Rows.allocate(T, cols, device=device) if fp8 else None
        self._rstd = torch.empty(T, dtype=torch.float32, device=device) if rstd else None
        self._shape = (T, cols, dtype, self.tensors[0].get_device())
        codes, scales = (None, None) if self._rows8 is None else self._rows8.tensors
        self._at = tuple(0 if t is None else t.data_ptr()
                         for t in (self._y, self._sum, codes, scales, self._rstd))

    y = property(lambda self: self._y)
    sum = property(lambda self: self._sum)
    rows8 = property(lambda self: self._rows8)
    rstd = property(lambda self: self._rstd)

    @property
    def tensors(self):
        more = () if self._rows8 is None else self._rows8.tensors
        return tuple(t for t in (self._y, self._sum, *more, self._rstd) if t is not None)

    @classmethod
    def allocate(cls, T: int, cols: int, dtype=torch.bfloat16, y: bool = True, sum: bool = False,
                 fp8: bool = False, rstd: bool = False, device="cuda") -> "NormBuffers":
        return cls(T, cols, dtype, device, y, sum, fp8, rstd)


def _norm_inputs(x, weight, residual, parts):
    """(device, T, cols, arguments up to the weight's type) of a norm's call."""
    dev, dtype = x.get_device(), x.dtype
    code = _HALF.get(dtype)
    if dev < 0 or code is None:
        cuda_device(x, "x")
        _half(x, "x")
    rows, cols, stride = rows_of(x, "x")
    if parts < 1 or rows % parts:
        raise ValueError(f"x has {rows} rows, no multiple of {parts} parts a token")
    T, pr, sr = rows // parts, 0, cols
    if residual is not None:
        if residual.dtype is not dtype or residual.shape != (T, cols):
            raise ValueError(f"residual must be {dtype} [{T}, {cols}], got {residual.dtype} "
                             f"{tuple(residual.shape)}")
        if residual.get_device() != dev:
            raise ValueError(f"residual is on {residual.device}, other buffers on cuda:{dev}")
        pr = residual.data_ptr()
        if not residual.is_contiguous():
            _, _, sr = rows_of(residual, "residual")
    pw, kind = _gain(weight, dtype, cols, dev)
    return dev, T, cols, (x.data_ptr(), code, stride, parts, pr, sr, T, cols, pw, kind)


def _gain(weight, dtype, cols, dev):
    kind = weight.dtype
    if kind is not dtype and kind is not torch.float32:
        raise ValueError(f"weight must be {dtype} or float32, got {kind}")
    if weight.numel() != cols:
        raise ValueError(f"weight holds {weight.numel()} elements, rows have {cols}")
    return need(weight, kind, cols, dev, "weight"), DTYPE_CODE[kind]


def moe_rms_norm(x, weight, eps, residual, parts, y, sum, codes, scales, rstd, stream=None) -> None:
    """The norm of ``residual`` (or None) plus the sum of each token's ``parts`` rows of ``x``
    [T * parts, cols] into caller-owned buffers, each of which may be None: y and sum [T, cols] of
    x's type, codes [T, cols] float8_e4m3fn with scales [T], rstd [T]."""
    dev, T, cols, args = _norm_inputs(x, weight, residual, parts)
    n = T * cols
    _norm(dev, stream, *args, eps, _optional(y, x.dtype, n, dev, "y"),
          _optional(sum, x.dtype, n, dev, "sum"), _optional(codes, FP8, n, dev, "codes"),
          _optional(scales, torch.float32, T, dev, "scales"),
          _optional(rstd, torch.float32, T, dev, "rstd"))


def rms_norm(x, weight, eps: float = 1e-6, residual=None, parts: int = 1, y: bool = True,
             sum: bool = False, fp8: bool = False, rstd: bool = False,
             out: Optional[NormBuffers] = None, stream=None) -> NormBuffers:
    """Run moe_rms_norm; allocates the outputs that are asked for unless ``out`` is given (whose
    buffers then say what is made).  A training step asks for ``sum`` and ``rstd``, which its
    gradient reads."""
    dev, T, cols, args = _norm_inputs(x, weight, residual, parts)
    if out is None:
        out = made(dev, stream, lambda: NormBuffers.allocate(T, cols, x.dtype, y, sum, fp8, rstd,
                                                             device=x.device))
    elif out._shape != (T, cols, x.dtype, dev):
        raise ValueError(f"out is for (T, cols, dtype, device) {out._shape}, the call is "
                         f"{(T, cols, x.dtype, dev)}")
    _norm(dev, stream, *args, eps, *out._at)
    return out


class NormGrads:
    """Gradients of the norm for one (T, cols): ``x`` [T, cols] of the rows' type, ``weight``
    [cols] float32 (None if not asked for), and their workspace."""

    __slots__ = ("_x", "_weight", "_workspace", "_shape")

    def __init__(self, T: int, cols: int, dtype, device, weight: bool):
        if dtype not in _HALF:
            raise ValueError(f"rows must be bfloat16 or float16, got {dtype}")
        ws = moe_rms_norm_backward_workspace_bytes(cols)
        if ws == 0:
            raise ValueError(f"invalid row length for the norm's gradient: {cols}")
        self._x = torch.empty(T, cols, dtype=dtype, device=device)
        self._weight = self._workspace = None
        if weight:
            self._weight = torch.empty(cols, dtype=torch.float32, device=device)
            self._workspace = torch.empty(ws, dtype=torch.uint8, device=device)
        self._shape = (T, cols, dtype, self._x.get_device())

    x = property(lambda self: self._x)
    weight = property(lambda self: self._weight)
    workspace = property(lambda self: self._workspace)

    @property
    def tensors(self):
        return (self._x,) if self._weight is None else (self._x, self._weight, self._workspace)

    @classmethod
    def allocate(cls, T: int, cols: int, dtype=torch.bfloat16, weight: bool = True,
                 device="cuda") -> "NormGrads":
        return cls(T, cols, dtype, device, weight)


def moe_rms_norm_backward(s, weight, rstd, grad, grad_rows, parts, grad_sum, grad_x, grad_weight,
                          workspace, stream=None) -> None:
    """Gradient of the norm into ``grad_x`` [T, cols] and ``grad_weight`` [cols] (None: not asked
    for, then without a workspace).  ``s`` and ``rstd`` are the forward call's; the gradient of its
    y is ``grad`` [T, cols] plus the sum of each token's ``parts`` rows of ``grad_rows``
    [T * parts, cols] (either may be None); ``grad_sum`` [T, cols] (or None) that of its sum."""
    dev = cuda_device(s, "s")
    code, dtype = _half(s, "s"), s.dtype
    if s.dim() != 2:
        raise ValueError("s must be [T, cols]")
    T, cols = s.shape
    n = T * cols
    pw, kind = _gain(weight, dtype, cols, dev)
    for t, name, rows in ((grad, "grad", T), (grad_rows, "grad_rows", T * parts),
                          (grad_sum, "grad_sum", T)):
        if t is not None and t.shape != (rows, cols):
            raise ValueError(f"{name} must be [{rows}, {cols}], got {tuple(t.shape)}")
    ws = (0, 0)
    if workspace is not None:
        ws = (need(workspace, torch.uint8, 0, dev, "workspace"), workspace.numel())
    _norm_backward(dev, stream, need(s, dtype, n, dev, "s"), code, pw, kind,
                   need(rstd, torch.float32, T, dev, "rstd"),
                   _optional(grad, dtype, n, dev, "grad"),
                   _optional(grad_rows, dtype, n * parts, dev, "grad_rows"), parts,
                   _optional(grad_sum, dtype, n, dev, "grad_sum"), T, cols,
                   need(grad_x, dtype, n, dev, "grad_x"),
                   _optional(grad_weight, torch.float32, cols, dev, "grad_weight"), *ws)


def rms_norm_backward(s, weight, rstd, grad=None, grad_rows=None, parts: int = 1, grad_sum=None,
                      weight_grad: bool = True, out: Optional[NormGrads] = None,
                      stream=None) -> NormGrads:
    """Allocate (unless ``out`` is given) and run moe_rms_norm_backward; returns the gradients."""
    if out is None:
        if s.dim() != 2:
            raise ValueError(f"s must be [T, cols], got {tuple(s.shape)}")
        out = made(cuda_device(s, "s"), stream,
                   lambda: NormGrads.allocate(*s.shape, s.dtype, weight_grad, device=s.device))
    elif out._shape != (*s.shape, s.dtype, s.get_device()):
        raise ValueError(f"out is for (T, cols, dtype, device) {out._shape}, the call is "
                         f"{(*s.shape, s.dtype, s.get_device())}")
    moe_rms_norm_backward(s, weight, rstd, grad, grad_rows, parts, grad_sum, out._x, out._weight,
                          out._workspace, stream)
    return out


# -------------------------------------------------------------------- the gated activation
def _gated_inputs(x, weights):
    dev = cuda_device(x, "x")
    code = _half(x, "x")
    rows, width, stride = rows_of(x, "x")
    if width % 2:
        raise ValueError(f"x must hold two halves side by side, got rows of {width}")
    if weights is not None and weights.numel() != rows:
        raise ValueError(f"weights holds {weights.numel()} elements, x has {rows} rows")
    return dev, code, rows, width // 2, stride, _optional(weights, torch.float32, rows, dev,
                                                          "weights")


def moe_swiglu(x, weights, y, codes, scales, stream=None) -> None:
    """The gated activation of ``x`` [rows, 2 * cols] times ``weights`` [rows] (or None) into y
    [rows, cols] and / or codes [rows, cols] float8_e4m3fn with scales [rows]."""
    dev, code, rows, cols, stride, pw = _gated_inputs(x, weights)
    n = rows * cols
    _gated(dev, stream, x.data_ptr(), code, stride, rows, cols, pw,
           _optional(y, x.dtype, n, dev, "y"), _optional(codes, FP8, n, dev, "codes"),
           _optional(scales, torch.float32, rows, dev, "scales"))


def swiglu(x, weights=None, fp8: bool = False, out=None, stream=None):
    """Run moe_swiglu; returns ``out`` (a tensor of x's type, or Fp8Rows), allocated unless given:
    Fp8Rows where ``fp8``.  ``weights`` are routing weights in route order (topk_weights)."""
    dev, code, rows, cols, stride, pw = _gated_inputs(x, weights)
    if out is None:
        out = made(dev, stream, lambda: Fp8Rows.allocate(rows, cols, device=x.device) if fp8 else
                   torch.empty(rows, cols, dtype=x.dtype, device=x.device))
    if isinstance(out, Fp8Rows):
        if out.lead != (rows,) or out.cols != cols or out.device != dev:
            raise ValueError(f"out holds rows of shape {tuple(out.codes.shape)} on "
                             f"cuda:{out.device}, the call makes {(rows, cols)} on cuda:{dev}")
        at = (0, out._codes.data_ptr(), out._scales.data_ptr())
    else:
        if out.shape != (rows, cols):
            raise ValueError(f"out must be {(rows, cols)}, got {tuple(out.shape)}")
        at = (need(out, x.dtype, rows * cols, dev, "out"), 0, 0)
    _gated(dev, stream, x.data_ptr(), code, stride, rows, cols, pw, *at)
    return out


def moe_swiglu_backward(grad, x, weights, grad_x, grad_weights, stream=None) -> None:
    """Gradient of the gated activation: ``grad`` [rows, cols] to ``grad_x`` [rows, 2 * cols] and
    ``grad_weights`` [rows] float32 (or None)."""
    dev, code, rows, cols, stride, pw = _gated_inputs(x, weights)
    if grad.shape != (rows, cols):
        raise ValueError(f"grad must be {(rows, cols)}, got {tuple(grad.shape)}")
    n = rows * cols
    _gated_backward(dev, stream, need(grad, x.dtype, n, dev, "grad"), x.data_ptr(), code, stride,
                    rows, cols, pw, need(grad_x, x.dtype, 2 * n, dev, "grad_x"),
                    _optional(grad_weights, torch.float32, rows, dev, "grad_weights"))


def swiglu_backward(grad, x, weights=None, out=None, stream=None):
    """Run moe_swiglu_backward; returns (grad_x, grad_weights), allocated unless ``out`` (the same
    pair) is given.  grad_weights is None without ``weights``; with them it is what
    ``route_backward`` takes, seen as [T, topk]."""
    if out is None:
        out = (made(cuda_device(x, "x"), stream, lambda: torch.empty(x.shape, dtype=x.dtype,
                                                                     device=x.device)),
               None if weights is None else
               made(cuda_device(x, "x"), stream, lambda: torch.empty(
                   weights.shape, dtype=torch.float32, device=x.device)))
    grad_x, grad_weights = out
    moe_swiglu_backward(grad, x, weights, grad_x, grad_weights, stream)
    return grad_x, grad_weights
