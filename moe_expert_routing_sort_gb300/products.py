"""The experts' products in 16 and 8 bits, driven by the sort step's metadata, and the gradients of
their rows and weights (see include/moe_route_sort.h).

``moe_*`` functions have the names of their C entry points and fill caller-owned buffers;
``experts_product``, ``experts_grad_rows`` and ``experts_grad_weights`` allocate what is not given.
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import load
from .marshal import Entry, cuda_device, made, need
from .rows import FP8, Fp8Rows

_product = Entry("moe_experts_product")
_grad_rows = Entry("moe_experts_grad_rows")
_grad_weights = Entry("moe_experts_grad_weights")

_CODE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, FP8: 3}
_HALF = (torch.bfloat16, torch.float16)


def moe_experts_product_workspace_bytes(T: int, E: int, topk: int, block_m: int) -> int:
    return int(load().moe_experts_product_workspace_bytes(T, E, topk, block_m))


class ProductWorkspace:
    """Workspace of the products and their gradients for one (T, E, topk, block_m), cleared when
    made.  It collects the DEVICE_* bits of the calls that it is given to; two calls that can run
    at the same time need one each."""

    __slots__ = ("_tensor",)

    def __init__(self, T: int, E: int, topk: int, block_m: int, device="cuda"):
        n = moe_experts_product_workspace_bytes(T, E, topk, block_m)
        if n == 0:
            raise ValueError("invalid shape for a products' workspace")
        self._tensor = torch.empty(n, dtype=torch.uint8, device=device)
        self._tensor[:4].zero_()

    tensor = property(lambda self: self._tensor)
    tensors = property(lambda self: (self._tensor,))

    @classmethod
    def allocate(cls, T: int, E: int, topk: int, block_m: int, device="cuda") -> "ProductWorkspace":
        return cls(T, E, topk, block_m, device)

    def status_word(self) -> int:
        """Device status bits of the completed calls so far (synchronises the device)."""
        torch.cuda.synchronize(self._tensor.device)
        return int(self._tensor[:4].view(torch.int32).item())

    def clear(self) -> None:
        """Clears the bits, in the order of the current stream."""
        self._tensor[:4].zero_()


def _list_args(T, E, topk, block_m, dev, sorted_token_ids, expert_ids, num_tokens_post_pad):
    """Addresses of the sorted list's ids, owners and length, checked for this shape."""
    n = T * topk
    P = n + min(n, E) * (block_m - 1)  # as moe_sort_max_padded
    return P, (need(sorted_token_ids, torch.int32, P, dev, "sorted_token_ids"),
               need(expert_ids, torch.int32, P // block_m if block_m > 0 else 0, dev,
                    "expert_ids"),
               need(num_tokens_post_pad, torch.int32, 1, dev, "num_tokens_post_pad"))


def _workspace(workspace, T, E, topk, block_m, dev, stream, like):
    if workspace is None:
        workspace = made(dev, stream, lambda: ProductWorkspace(T, E, topk, block_m,
                                                               device=like.device))
    if isinstance(workspace, ProductWorkspace):
        workspace = workspace.tensor
    return workspace, (need(workspace, torch.uint8, 0, dev, "workspace"), workspace.numel())


def _rows(x, name, T, topk, cols, dtype, dev):
    """(address, whether a row is a route's) of 16-bit rows [T or T * topk, cols]."""
    if x.dim() != 2 or x.shape[1] != cols or x.shape[0] not in (T, T * topk):
        raise ValueError(f"{name} must be [T = {T} or T * topk = {T * topk}, {cols}], got "
                         f"{tuple(x.shape)}")
    return need(x, dtype, 0, dev, name), 0 if x.shape[0] == T else 1


def _three(name, w):
    if w.dim() != 3:
        raise ValueError(f"{name} must be [E, outs, cols], got {tuple(w.shape)}")


def _half_weights(w):
    dev = cuda_device(w, "w")
    if w.dtype not in _HALF:
        raise ValueError(f"w must be bfloat16 or float16, got {w.dtype}")
    _three("w", w)
    return dev, need(w, w.dtype, 0, dev, "w")


def _out(out, shape, kinds, dev, name):
    if out.dtype not in kinds:
        raise ValueError(f"{name} must be one of {', '.join(map(str, kinds))}, got {out.dtype}")
    if tuple(out.shape) != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(out.shape)}")
    return need(out, out.dtype, 0, dev, name), _CODE[out.dtype]


def moe_experts_product(x, w, T, topk, block_m, sorted_token_ids, sorted_weights, expert_ids,
                        num_tokens_post_pad, out, workspace, stream=None) -> None:
    """Products of rows with their experts' weights into ``out`` [T * topk, outs] (bfloat16,
    float16 or float32; row r is route r).  ``x`` has T rows (one per token) or T * topk (one per
    route), ``w`` is [E, outs, cols]: tensors of one 16-bit type, or both Fp8Rows.  The sorted list
    is that of moe_sort or moe_route_sort; ``sorted_weights`` may be None (rows are not scaled)."""
    if isinstance(w, Fp8Rows):
        if not isinstance(x, Fp8Rows):
            raise ValueError("x must be Fp8Rows where w is")
        dev = w.device
        if len(x.lead) != 1 or len(w.lead) != 2 or x.cols != w.cols:
            raise ValueError(f"x must be [rows, cols] and w [E, outs, cols], got "
                             f"{(*x.lead, x.cols)} and {(*w.lead, w.cols)}")
        if x.device != dev:
            raise ValueError(f"x is on cuda:{x.device}, w on cuda:{dev}")
        (E, outs), cols, rows = w.lead, w.cols, x.lead[0]
        if rows != T and rows != T * topk:
            raise ValueError(f"x must have T = {T} or T * topk = {T * topk} rows, got {rows}")
        px, xs, per = x._codes.data_ptr(), x._scales.data_ptr(), 0 if rows == T else 1
        pw, ws, kind = w._codes.data_ptr(), w._scales.data_ptr(), 3
    else:
        dev, pw = _half_weights(w)
        E, outs, cols = w.shape
        if isinstance(x, Fp8Rows):
            raise ValueError("x must be a tensor of w's type")
        px, per = _rows(x, "x", T, topk, cols, w.dtype, dev)
        xs, ws, kind = 0, 0, _CODE[w.dtype]
    P, (ids, owners, length) = _list_args(T, E, topk, block_m, dev, sorted_token_ids, expert_ids,
                                          num_tokens_post_pad)
    _, at = _workspace(workspace, T, E, topk, block_m, dev, stream, out)
    _product(dev, stream, px, kind, xs, per, pw, ws, T, E, topk, cols, outs, block_m, ids,
             0 if sorted_weights is None else need(sorted_weights, torch.float32, P, dev,
                                                   "sorted_weights"),
             owners, length,
             *_out(out, (T * topk, outs), (*_HALF, torch.float32), dev, "out"), *at)


def experts_product(x, w, T: int, topk: int, block_m: int, sorted_token_ids, expert_ids,
                    num_tokens_post_pad, sorted_weights=None, dtype=None,
                    out: Optional[torch.Tensor] = None, workspace=None,
                    stream=None) -> torch.Tensor:
    """Run moe_experts_product on rows ``x`` and weights ``w`` [E, outs, cols]; returns ``out``
    [T * topk, outs], of type ``dtype`` (that of 16-bit rows, bfloat16 for Fp8Rows).  Without
    ``out`` the rows of dropped routes are zero: a new buffer is cleared first, a pass over it that
    a call with ``out`` saves.  Without ``workspace`` (a ProductWorkspace, or a tensor, see
    moe_experts_product_workspace_bytes) one is made, and its status bits are lost."""
    if out is None:
        eight = isinstance(w, Fp8Rows)
        dev, like = (w.device, w.codes) if eight else (cuda_device(w, "w"), w)
        _three("w", like)
        kind = dtype or (torch.bfloat16 if eight else w.dtype)
        out = made(dev, stream, lambda: torch.zeros(T * topk, like.shape[1], dtype=kind,
                                                    device=like.device))
    moe_experts_product(x, w, T, topk, block_m, sorted_token_ids, sorted_weights, expert_ids,
                        num_tokens_post_pad, out, workspace, stream)
    return out


def moe_experts_grad_rows(grad, w, T, topk, block_m, sorted_token_ids, expert_ids,
                          num_tokens_post_pad, grad_rows, workspace, stream=None) -> None:
    """Gradient of the product's rows into ``grad_rows`` [T * topk, cols], one row a route (of rows
    of x shared by a token's routes: the sum of topk adjacent rows).  ``grad`` has T or T * topk
    rows of outs elements, ``w`` is [E, outs, cols], both of one 16-bit type."""
    dev, pw = _half_weights(w)
    E, outs, cols = w.shape
    pg, per = _rows(grad, "grad", T, topk, outs, w.dtype, dev)
    _, lists = _list_args(T, E, topk, block_m, dev, sorted_token_ids, expert_ids,
                          num_tokens_post_pad)
    _, at = _workspace(workspace, T, E, topk, block_m, dev, stream, grad_rows)
    _grad_rows(dev, stream, pg, _CODE[w.dtype], per, pw, T, E, topk, cols, outs, block_m, *lists,
               *_out(grad_rows, (T * topk, cols), (*_HALF, torch.float32), dev, "grad_rows"), *at)


def experts_grad_rows(grad, w, T: int, topk: int, block_m: int, sorted_token_ids, expert_ids,
                      num_tokens_post_pad, dtype=None, out: Optional[torch.Tensor] = None,
                      workspace=None, stream=None) -> torch.Tensor:
    """Run moe_experts_grad_rows; returns ``out`` [T * topk, cols], of type ``dtype`` (w's).
    Without ``out`` the rows of dropped routes are zero."""
    if out is None:
        _three("w", w)
        out = made(cuda_device(w, "w"), stream,
                   lambda: torch.zeros(T * topk, w.shape[-1], dtype=dtype or w.dtype,
                                       device=w.device))
    moe_experts_grad_rows(grad, w, T, topk, block_m, sorted_token_ids, expert_ids,
                          num_tokens_post_pad, out, workspace, stream)
    return out


def moe_experts_grad_weights(grad, x, T, topk, block_m, sorted_token_ids, expert_ids,
                             num_tokens_post_pad, grad_weights, workspace, stream=None) -> None:
    """Gradient of the product's weights into ``grad_weights`` [E, outs, cols] (the rows' type or
    float32), every element of it.  ``grad`` has T or T * topk rows of outs elements, ``x`` T or
    T * topk of cols, both of one 16-bit type."""
    dev = cuda_device(grad_weights, "grad_weights")
    _three("grad_weights", grad_weights)
    E, outs, cols = grad_weights.shape
    if grad.dtype not in _HALF:
        raise ValueError(f"grad must be bfloat16 or float16, got {grad.dtype}")
    pg, gper = _rows(grad, "grad", T, topk, outs, grad.dtype, dev)
    px, xper = _rows(x, "x", T, topk, cols, grad.dtype, dev)
    _, lists = _list_args(T, E, topk, block_m, dev, sorted_token_ids, expert_ids,
                          num_tokens_post_pad)
    _, at = _workspace(workspace, T, E, topk, block_m, dev, stream, grad_weights)
    _grad_weights(dev, stream, pg, _CODE[grad.dtype], gper, px, xper, T, E, topk, cols, outs,
                  block_m, *lists,
                  *_out(grad_weights, (E, outs, cols), (grad.dtype, torch.float32), dev,
                        "grad_weights"), *at)


def experts_grad_weights(grad, x, E: int, T: int, topk: int, block_m: int, sorted_token_ids,
                         expert_ids, num_tokens_post_pad, dtype=torch.float32,
                         out: Optional[torch.Tensor] = None, workspace=None,
                         stream=None) -> torch.Tensor:
    """Run moe_experts_grad_weights; returns ``out`` [E, outs, cols], of type ``dtype``."""
    if out is None:
        if grad.dim() != 2 or x.dim() != 2:
            raise ValueError(f"grad and x must be matrices, got {tuple(grad.shape)} and "
                             f"{tuple(x.shape)}")
        out = made(cuda_device(grad, "grad"), stream,
                   lambda: torch.empty(E, grad.shape[-1], x.shape[-1], dtype=dtype,
                                       device=grad.device))
    elif out.dim() > 0 and out.shape[0] != E:
        raise ValueError(f"out must be of {E} experts, got {tuple(out.shape)}")
    moe_experts_grad_weights(grad, x, T, topk, block_m, sorted_token_ids, expert_ids,
                             num_tokens_post_pad, out, workspace, stream)
    return out
