"""The experts' products in microscaled 4-bit floating point (MXFP4), driven by the sort step's
metadata, with the quantisation of rows and weights (see include/moe_route_sort.h).

``moe_*`` functions have the names of their C entry points and fill caller-owned buffers;
``mxfp4_quantize``, ``mxfp4_dequantize`` and ``experts_mxfp4`` allocate what is not given.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from .binding import _sort_sizes, load
from .marshal import DTYPE_CODE, cuda_device, launch, need, rows_of


def moe_mxfp4_scale_cols(cols: int) -> int:
    return int(load().moe_mxfp4_scale_cols(cols))


def moe_experts_mxfp4_workspace_bytes(T: int, E: int, topk: int, block_m: int) -> int:
    return int(load().moe_experts_mxfp4_workspace_bytes(T, E, topk, block_m))


@dataclass
class Mxfp4Rows:
    """MXFP4 rows: ``codes`` [..., cols / 2] and ``scales`` [..., moe_mxfp4_scale_cols(cols)],
    both uint8.  Weights of E experts are [E, outs, ...]."""

    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def cols(self) -> int:
        return 2 * self.codes.shape[-1]

    @classmethod
    def allocate(cls, rows, cols: int, device="cuda") -> "Mxfp4Rows":
        """Room for ``rows`` (a number, or a tuple such as (E, outs)) of ``cols`` elements."""
        lead = tuple(rows) if isinstance(rows, (tuple, list)) else (rows,)
        sc = moe_mxfp4_scale_cols(cols)
        if sc == 0:
            raise ValueError(f"cols must be a multiple of 32 in [32, 32768], got {cols}")
        return cls(torch.empty(*lead, cols // 2, dtype=torch.uint8, device=device),
                   torch.empty(*lead, sc, dtype=torch.uint8, device=device))


def moe_mxfp4_quantize(x, codes, scales, stream=None) -> None:
    """Rows of ``x`` (a matrix with dense rows: bfloat16, float16 or float32) into codes and
    scales."""
    dev = cuda_device(x, "x")
    if x.dtype not in DTYPE_CODE:
        raise ValueError(f"x must be bfloat16, float16 or float32, got {x.dtype}")
    rows, cols, stride = rows_of(x, "x")
    launch("moe_mxfp4_quantize", dev, stream, x.data_ptr(), DTYPE_CODE[x.dtype], rows, cols,
           stride, need(codes, torch.uint8, rows * (cols // 2), dev, "codes"),
           need(scales, torch.uint8, rows * ((cols + 127) // 128 * 4), dev, "scales"))


def mxfp4_quantize(x, out: Optional[Mxfp4Rows] = None, stream=None) -> Mxfp4Rows:
    """Quantise the rows of ``x`` ([..., cols]); allocates the result unless ``out`` is given."""
    if out is None:
        out = Mxfp4Rows.allocate(x.shape[:-1], x.shape[-1], device=x.device)
    elif out.codes.shape[:-1] != x.shape[:-1] or out.cols != x.shape[-1]:
        raise ValueError(f"out holds rows of shape {tuple(out.codes.shape)}, x is "
                         f"{tuple(x.shape)}")
    moe_mxfp4_quantize(x if x.dim() == 2 else x.reshape(-1, x.shape[-1]), out.codes, out.scales,
                       stream=stream)
    return out


def moe_mxfp4_dequantize(codes, scales, y, stream=None) -> None:
    """The values that codes and scales stand for into ``y`` (a matrix with dense rows, bfloat16
    or float32)."""
    dev = cuda_device(y, "y")
    if y.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"y must be bfloat16 or float32, got {y.dtype}")
    rows, cols, stride = rows_of(y, "y")
    launch("moe_mxfp4_dequantize", dev, stream,
           need(codes, torch.uint8, rows * (cols // 2), dev, "codes"),
           need(scales, torch.uint8, rows * ((cols + 127) // 128 * 4), dev, "scales"), rows, cols,
           y.data_ptr(), DTYPE_CODE[y.dtype], stride)


def mxfp4_dequantize(rows: Mxfp4Rows, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """The values of ``rows`` as a tensor [..., cols]; allocates it unless ``out`` is given."""
    shape = (*rows.codes.shape[:-1], rows.cols)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=rows.codes.device)
    elif out.shape != shape:
        raise ValueError(f"out is {tuple(out.shape)}, the rows are {shape}")
    y = out if out.dim() == 2 else out.view(-1, rows.cols)
    moe_mxfp4_dequantize(rows.codes, rows.scales, y, stream=stream)
    return out


def moe_experts_mxfp4(x_codes, x_scales, w_codes, w_scales, T, topk, block_m, sorted_token_ids,
                      sorted_weights, expert_ids, num_tokens_post_pad, out, workspace,
                      stream=None) -> None:
    """Products of MXFP4 rows with their experts' MXFP4 weights, into ``out`` [T * topk, outs]
    (bfloat16 or float32; row r is route r).  ``x_codes`` has T rows (one per token) or T * topk
    (one per route); ``w_codes`` is [E, outs, cols / 2]; the sorted list is that of moe_sort or
    moe_route_sort; ``sorted_weights`` may be None (rows are not scaled)."""
    dev = cuda_device(x_codes, "x_codes")
    if x_codes.dim() != 2 or w_codes.dim() != 3 or x_codes.shape[1] != w_codes.shape[2]:
        raise ValueError("x_codes must be [rows, cols / 2] and w_codes [E, outs, cols / 2]")
    (xr, half), (E, outs) = x_codes.shape, w_codes.shape[:2]
    if xr != T and xr != T * topk:
        raise ValueError(f"x_codes must have T = {T} or T * topk = {T * topk} rows, got {xr}")
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out must be bfloat16 or float32, got {out.dtype}")
    cols = 2 * half
    sc = (cols + 127) // 128 * 4
    P, NB = _sort_sizes(T, E, topk, block_m)
    launch("moe_experts_mxfp4", dev, stream,
           need(x_codes, torch.uint8, xr * half, dev, "x_codes"),
           need(x_scales, torch.uint8, xr * sc, dev, "x_scales"), int(xr != T),
           need(w_codes, torch.uint8, E * outs * half, dev, "w_codes"),
           need(w_scales, torch.uint8, E * outs * sc, dev, "w_scales"), T, E, topk, cols, outs,
           block_m, need(sorted_token_ids, torch.int32, P, dev, "sorted_token_ids"),
           None if sorted_weights is None else need(sorted_weights, torch.float32, P, dev,
                                                    "sorted_weights"),
           need(expert_ids, torch.int32, NB, dev, "expert_ids"),
           need(num_tokens_post_pad, torch.int32, 1, dev, "num_tokens_post_pad"),
           need(out, out.dtype, T * topk * outs, dev, "out"), DTYPE_CODE[out.dtype],
           need(workspace, torch.uint8, 0, dev, "workspace"), workspace.numel())


def experts_mxfp4(x: Mxfp4Rows, w: Mxfp4Rows, T: int, topk: int, block_m: int, sorted_token_ids,
                  expert_ids, num_tokens_post_pad, sorted_weights=None, dtype=torch.bfloat16,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Run moe_experts_mxfp4; returns ``out`` [T * topk, outs].  Without ``out`` the rows of
    dropped routes are zero (a new buffer is cleared first)."""
    if out is None:
        out = torch.zeros(T * topk, w.codes.shape[1], dtype=dtype, device=w.codes.device)
    if workspace is None:
        workspace = torch.zeros(moe_experts_mxfp4_workspace_bytes(T, w.codes.shape[0], topk,
                                                                  block_m),
                                dtype=torch.uint8, device=w.codes.device)
    moe_experts_mxfp4(x.codes, x.scales, w.codes, w.scales, T, topk, block_m, sorted_token_ids,
                      sorted_weights, expert_ids, num_tokens_post_pad, out, workspace,
                      stream=stream)
    return out
