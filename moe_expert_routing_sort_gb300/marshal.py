"""Argument checks and launch helpers shared by the training and experts bindings."""
from __future__ import annotations

import contextlib

import torch

from .binding import _check, load

# type codes of include/moe_route_sort.h
DTYPE_CODE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

_here = contextlib.nullcontext()


def need(t: torch.Tensor, dtype, numel: int, device: torch.device, name: str) -> int:
    """Checks one dense device buffer of at least ``numel`` elements; returns its address."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other buffers on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements; this shape needs {numel}")
    return t.data_ptr()


def cuda_device(t: torch.Tensor, name: str) -> torch.device:
    """The CUDA device of the call's first tensor, which the others are checked against."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def rows_of(t: torch.Tensor, name: str):
    """(rows, cols, elements between rows) of a matrix whose rows are dense."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got {tuple(t.shape)}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have dense rows")
    return rows, cols, (t.stride(0) if rows > 1 else cols)


def launch(name: str, device: torch.device, stream, *args) -> None:
    """Calls C entry point ``name`` with ``device`` current on ``stream`` (None: the device's
    current stream) and raises on a negative status."""
    other = torch.cuda.current_device() != device.index
    with torch.cuda.device(device) if other else _here:
        if stream is None:
            handle = torch.cuda.current_stream(device).cuda_stream
        else:
            handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        rc = getattr(load(), name)(*args, handle)
    if rc:
        _check(rc, name)
