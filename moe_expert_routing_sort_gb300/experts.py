"""The experts' products in microscaled 4-bit floating point (MXFP4), driven by the sort step's
metadata, with the quantisation of rows and weights (see include/moe_route_sort.h).

``moe_*`` functions have the names of their C entry points and fill caller-owned buffers;
``mxfp4_quantize``, ``mxfp4_dequantize`` and ``experts_mxfp4`` allocate what is not given.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from .binding import _check, load
from .marshal import DTYPE_CODE, Entry, cuda_device, made, need, rows_of, stream_handle

_quantize = Entry("moe_mxfp4_quantize")
_dequantize = Entry("moe_mxfp4_dequantize")
_experts = Entry("moe_experts_mxfp4")


def moe_mxfp4_scale_cols(cols: int) -> int:
    return int(load().moe_mxfp4_scale_cols(cols))


def moe_experts_mxfp4_workspace_bytes(T: int, E: int, topk: int, block_m: int) -> int:
    return int(load().moe_experts_mxfp4_workspace_bytes(T, E, topk, block_m))


def _scale_cols(cols: int) -> int:
    return (cols + 127) // 128 * 4


class Mxfp4Rows:
    """MXFP4 rows: ``codes`` [..., cols / 2] and ``scales`` [..., moe_mxfp4_scale_cols(cols)],
    both uint8 on one CUDA device.  Weights of E experts are [E, outs, ...].  The two tensors are
    checked here, once, and cannot be exchanged afterwards."""

    __slots__ = ("_codes", "_scales", "lead", "cols", "device")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        self.device = cuda_device(codes, "codes")
        self._codes, self._scales = codes, scales
        self.lead = tuple(codes.shape[:-1])   # (rows,), or (E, outs)
        self.cols = 2 * codes.shape[-1]
        if tuple(scales.shape) != (*self.lead, _scale_cols(self.cols)):
            raise ValueError(f"scales must be {(*self.lead, _scale_cols(self.cols))} for codes "
                             f"{tuple(codes.shape)}, got {tuple(scales.shape)}")
        need(codes, torch.uint8, 0, self.device, "codes")
        need(scales, torch.uint8, 0, self.device, "scales")

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    tensors = property(lambda self: (self._codes, self._scales))

    @classmethod
    def allocate(cls, rows, cols: int, device="cuda") -> "Mxfp4Rows":
        """Room for ``rows`` (a number, or a tuple such as (E, outs)) of ``cols`` elements."""
        lead = tuple(rows) if isinstance(rows, (tuple, list)) else (rows,)
        sc = moe_mxfp4_scale_cols(cols)
        if sc == 0:
            raise ValueError(f"cols must be a multiple of 32 in [32, 32768], got {cols}")
        return cls(torch.empty(*lead, cols // 2, dtype=torch.uint8, device=device),
                   torch.empty(*lead, sc, dtype=torch.uint8, device=device))


class ExpertsPlan(NamedTuple):
    """How a product is divided: outputs of a tile, blocks of a window (1: blocks by themselves),
    parts of a block, tiles along the outputs, tiles of a unit, units along the outputs, steps of
    256 columns."""

    tile_outs: int
    window: int
    parts: int
    tiles: int
    unit_tiles: int
    units: int
    steps: int


def moe_experts_mxfp4_plan(T: int, E: int, topk: int, cols: int, outs: int, block_m: int,
                           sms: int = 152) -> ExpertsPlan:
    plan = (ctypes.c_int32 * 7)()
    _check(load().moe_experts_mxfp4_plan(T, E, topk, cols, outs, block_m, sms, plan),
           "moe_experts_mxfp4_plan")
    return ExpertsPlan(*plan)


class ExpertsWorkspace:
    """Workspace of the experts' products for one (T, E, topk, block_m), cleared when made.  It
    collects the DEVICE_* bits of the calls that it is given to, which may run at the same time."""

    __slots__ = ("tensor",)

    def __init__(self, T: int, E: int, topk: int, block_m: int, device="cuda"):
        n = moe_experts_mxfp4_workspace_bytes(T, E, topk, block_m)
        if n == 0:
            raise ValueError("invalid shape for an experts' workspace")
        self.tensor = torch.zeros(n, dtype=torch.uint8, device=device)

    @classmethod
    def allocate(cls, T: int, E: int, topk: int, block_m: int, device="cuda") -> "ExpertsWorkspace":
        return cls(T, E, topk, block_m, device)

    def status_word(self) -> int:
        """Device status bits of the completed calls so far (synchronises the device)."""
        torch.cuda.synchronize(self.tensor.device)
        return int(self.tensor[:4].view(torch.int32).item())

    def clear(self) -> None:
        """Clears the bits, in the order of the current stream."""
        self.tensor.zero_()


def moe_experts_mxfp4_status(dst, clear: bool = False, stream=None) -> None:
    """Copy the status bits of the products without a workspace on dst's device into dst[0] (an
    int32 CUDA tensor), and clear them if asked, enqueued on the stream."""
    dev = cuda_device(dst, "dst")
    address = need(dst, torch.int32, 1, dev, "dst")
    with torch.cuda.device(dev):
        rc = load().moe_experts_mxfp4_status(address, 1 if clear else 0, stream_handle(dev, stream))
    _check(rc, "moe_experts_mxfp4_status")


def experts_status(device="cuda", clear: bool = False) -> int:
    """Device status bits (DEVICE_*; 0: nothing to report) of the products on ``device`` that were
    given no workspace, since they were last cleared (synchronises the device)."""
    dst = torch.empty(1, dtype=torch.int32, device=device)
    torch.cuda.synchronize(dst.device)
    moe_experts_mxfp4_status(dst, clear, stream=torch.cuda.current_stream(dst.device))
    return int(dst.item())


def moe_mxfp4_quantize(x, codes, scales, stream=None) -> None:
    """Rows of ``x`` (a matrix with dense rows: bfloat16, float16 or float32) into codes and
    scales."""
    dev = cuda_device(x, "x")
    if x.dtype not in DTYPE_CODE:
        raise ValueError(f"x must be bfloat16, float16 or float32, got {x.dtype}")
    rows, cols, stride = rows_of(x, "x")
    _quantize(dev, stream, x.data_ptr(), DTYPE_CODE[x.dtype], rows, cols, stride,
              need(codes, torch.uint8, rows * (cols // 2), dev, "codes"),
              need(scales, torch.uint8, rows * _scale_cols(cols), dev, "scales"))


def mxfp4_quantize(x, out: Optional[Mxfp4Rows] = None, stream=None) -> Mxfp4Rows:
    """Quantise the rows of ``x`` ([..., cols]); allocates the result unless ``out`` is given."""
    dev = cuda_device(x, "x")
    code = DTYPE_CODE.get(x.dtype)
    if code is None:
        raise ValueError(f"x must be bfloat16, float16 or float32, got {x.dtype}")
    shape = x.shape
    if out is None:
        out = made(dev, stream, lambda: Mxfp4Rows.allocate(shape[:-1], shape[-1], device=x.device))
    elif out.lead != shape[:-1] or out.cols != shape[-1] or out.device != dev:
        raise ValueError(f"out holds rows of shape {tuple(out.codes.shape)} on cuda:{out.device}, "
                         f"x is {tuple(shape)} on {x.device}")
    if len(shape) != 2:
        given = x
        x = made(dev, stream, lambda: given.reshape(-1, shape[-1]))  # a copy, if not a view
    rows, cols, stride = rows_of(x, "x")
    _quantize(dev, stream, x.data_ptr(), code, rows, cols, stride, out._codes.data_ptr(),
              out._scales.data_ptr())
    return out


def moe_mxfp4_dequantize(codes, scales, y, stream=None) -> None:
    """The values that codes and scales stand for into ``y`` (a matrix with dense rows, bfloat16
    or float32)."""
    dev = cuda_device(y, "y")
    if y.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"y must be bfloat16 or float32, got {y.dtype}")
    rows, cols, stride = rows_of(y, "y")
    _dequantize(dev, stream, need(codes, torch.uint8, rows * (cols // 2), dev, "codes"),
                need(scales, torch.uint8, rows * _scale_cols(cols), dev, "scales"), rows, cols,
                y.data_ptr(), DTYPE_CODE[y.dtype], stride)


def mxfp4_dequantize(rows: Mxfp4Rows, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """The values of ``rows`` as a tensor [..., cols]; allocates it unless ``out`` is given."""
    dev, cols = rows.device, rows.cols
    if out is None:
        out = made(dev, stream, lambda: torch.empty((*rows.lead, cols), dtype=dtype,
                                                    device=rows.codes.device))
    elif out.shape != (*rows.lead, cols) or out.get_device() != dev:
        raise ValueError(f"out is {tuple(out.shape)} on {out.device}, the rows are "
                         f"{(*rows.lead, cols)} on cuda:{dev}")
    kind = out.dtype
    if kind is not torch.bfloat16 and kind is not torch.float32:
        raise ValueError(f"out must be bfloat16 or float32, got {kind}")
    n, _, stride = rows_of(out if out.dim() == 2 else out.view(-1, cols), "out")
    _dequantize(dev, stream, rows._codes.data_ptr(), rows._scales.data_ptr(), n, cols,
                out.data_ptr(), DTYPE_CODE[kind], stride)
    return out


def _list_args(T, E, topk, block_m, outs, dev, sorted_token_ids, sorted_weights, expert_ids,
               num_tokens_post_pad, out, workspace):
    """Addresses of the sorted list, the output and the workspace, checked for this shape."""
    kind = out.dtype
    if kind is not torch.bfloat16 and kind is not torch.float32:
        raise ValueError(f"out must be bfloat16 or float32, got {kind}")
    n = T * topk
    P = n + min(n, E) * (block_m - 1)  # as moe_sort_max_padded
    return (need(sorted_token_ids, torch.int32, P, dev, "sorted_token_ids"),
            0 if sorted_weights is None else need(sorted_weights, torch.float32, P, dev,
                                                     "sorted_weights"),
            need(expert_ids, torch.int32, P // block_m if block_m > 0 else 0, dev, "expert_ids"),
            need(num_tokens_post_pad, torch.int32, 1, dev, "num_tokens_post_pad"),
            need(out, kind, n * outs, dev, "out"), DTYPE_CODE[kind],
            *((0, 0) if workspace is None else
              (need(workspace, torch.uint8, 0, dev, "workspace"), workspace.numel())))


def moe_experts_mxfp4(x_codes, x_scales, w_codes, w_scales, T, topk, block_m, sorted_token_ids,
                      sorted_weights, expert_ids, num_tokens_post_pad, out, workspace,
                      stream=None) -> None:
    """Products of MXFP4 rows with their experts' MXFP4 weights, into ``out`` [T * topk, outs]
    (bfloat16 or float32; row r is route r).  ``x_codes`` has T rows (one per token) or T * topk
    (one per route); ``w_codes`` is [E, outs, cols / 2]; the sorted list is that of moe_sort or
    moe_route_sort; ``sorted_weights`` may be None (rows are not scaled), ``workspace`` too (the
    status bits are then those of moe_experts_mxfp4_status)."""
    experts_mxfp4(Mxfp4Rows(x_codes, x_scales), Mxfp4Rows(w_codes, w_scales), T, topk, block_m,
                  sorted_token_ids, expert_ids, num_tokens_post_pad, sorted_weights, out=out,
                  workspace=workspace, stream=stream)


def experts_mxfp4(x: Mxfp4Rows, w: Mxfp4Rows, T: int, topk: int, block_m: int, sorted_token_ids,
                  expert_ids, num_tokens_post_pad, sorted_weights=None, dtype=torch.bfloat16,
                  out: Optional[torch.Tensor] = None, workspace=None,
                  stream=None) -> torch.Tensor:
    """Run moe_experts_mxfp4 on rows ``x`` and weights ``w`` [E, outs, ...]; returns ``out``
    [T * topk, outs].  Without ``out`` the rows of dropped routes are zero: a new buffer is
    cleared first, a pass over it that a call with ``out`` saves.

    A bad expert id or a device wait that gave up shows in the status bits alone: of
    ``workspace`` (an ExpertsWorkspace, or a tensor, see moe_experts_mxfp4_workspace_bytes), or,
    without one, of ``experts_status(device)``."""
    dev = w.device
    if len(x.lead) != 1 or len(w.lead) != 2 or x.cols != w.cols:
        raise ValueError(f"x must be [rows, cols] and w [E, outs, cols], got {(*x.lead, x.cols)} "
                         f"and {(*w.lead, w.cols)}")
    if x.device != dev:
        raise ValueError(f"x is on cuda:{x.device}, w on cuda:{dev}")
    (xr,), (E, outs) = x.lead, w.lead
    if xr != T and xr != T * topk:
        raise ValueError(f"x must have T = {T} or T * topk = {T * topk} rows, got {xr}")
    if out is None:
        out = made(dev, stream, lambda: torch.zeros(T * topk, outs, dtype=dtype,
                                                    device=w.codes.device))
    if isinstance(workspace, ExpertsWorkspace):
        workspace = workspace.tensor
    _experts(dev, stream, x._codes.data_ptr(), x._scales.data_ptr(), 0 if xr == T else 1,
             w._codes.data_ptr(), w._scales.data_ptr(), T, E, topk, x.cols, outs, block_m,
             *_list_args(T, E, topk, block_m, outs, dev, sorted_token_ids, sorted_weights,
                         expert_ids, num_tokens_post_pad, out, workspace))
    return out
