"""Argument checks and the launch of C entry points shared by the training and experts bindings.

A call of these operators can take less time on the GPU than its checks take here, so a check asks
each tensor for as little as it can, and containers check their own tensors once.
"""
from __future__ import annotations

import struct

import torch

from .binding import _check, load

# type codes of include/moe_route_sort.h
DTYPE_CODE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

# (the call behind torch.cuda.current_device, which a tensor of a call has initialised CUDA for)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# (a torch without CUDA has none, nor tensors for a call that wants it)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def need(t: torch.Tensor, dtype, numel: int, device: int, name: str) -> int:
    """Checks one dense buffer of at least ``numel`` elements on CUDA device ``device``; returns
    its address."""
    if (t.dtype is dtype and t.get_device() == device and t.is_contiguous()
            and t.numel() >= numel):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, other buffers on cuda:{device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} holds {t.numel()} elements; this shape needs {numel}")


def cuda_device(t: torch.Tensor, name: str) -> int:
    """The CUDA device of the call's first tensor, which the others are checked against."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def made(device: int, stream, make):
    """What ``make()`` allocates for a call on ``stream``: made on that stream, so that what fills
    it, and what had its memory before, is over when the call runs.  The caller's current stream is
    recorded on it, where it may be used and let go."""
    if stream is None:
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)),
                                           device=device)
    current = torch.cuda.current_stream(device)
    if current == stream:
        return make()
    with torch.cuda.stream(stream):
        got = make()
    for t in getattr(got, "tensors", (got,)):
        t.record_stream(current)
    return got


def stream_handle(device: int, stream) -> int:
    """Address of ``stream`` (a stream or an address), or of the device's current one."""
    if stream is None:
        return _raw_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def rows_of(t: torch.Tensor, name: str):
    """(rows, cols, elements between rows) of a matrix whose rows are dense."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got {tuple(t.shape)}")
    rows, cols = t.shape
    stride, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must have dense rows")
    return rows, cols, (stride if rows > 1 else cols)


# The operations' numbers and arguments (include/moe_route_sort.h): q an address, an integer or the
# stream, d a float.
_OPERATIONS = {
    "moe_balance_loss": (1, "8qd6q"),
    "moe_route_backward": (2, "11q2d3q"),
    "moe_mxfp4_quantize": (3, "8q"),
    "moe_mxfp4_dequantize": (4, "8q"),
    "moe_experts_mxfp4": (5, "20q"),
    "moe_fp8_quantize": (6, "8q"),
    "moe_rms_norm": (7, "10qd6q"),
    "moe_rms_norm_backward": (8, "16q"),
    "moe_swiglu": (9, "10q"),
    "moe_swiglu_backward": (10, "10q"),
    "moe_experts_product": (11, "21q"),
    "moe_experts_grad_rows": (12, "18q"),
    "moe_experts_grad_weights": (13, "19q"),
}


class Entry:
    """C entry point ``name``, called with its device current and the stream as last argument;
    raises on a negative status.  The arguments go as one array (moe_call_packed): converting 20
    of them one by one takes longer than the smallest kernels.  A NULL is 0."""

    __slots__ = ("name", "op", "count", "pack", "fn")

    def __init__(self, name: str):
        self.name = name
        self.op, args = _OPERATIONS[name]
        self.pack = struct.Struct("=qq" + args).pack
        self.count = (struct.calcsize("=" + args)) // 8
        self.fn = None

    def __call__(self, device: int, stream, *args) -> None:
        fn = self.fn
        if fn is None:
            fn = self.fn = load().moe_call_packed
        packed = self.pack(self.op, self.count, *args,
                           _raw_stream(device) if stream is None else stream_handle(device, stream))
        if _current_device() == device:
            rc = fn(packed)
        else:
            with torch.cuda.device(device):
                rc = fn(packed)
        if rc:
            _check(rc, self.name)
