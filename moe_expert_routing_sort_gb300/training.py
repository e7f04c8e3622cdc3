"""Training a router: its balance loss with per-expert counts, and the gradient of the routing
weights and of that loss to the logits (see include/moe_route_sort.h).

``moe_*`` functions have the names of their C entry points and fill caller-owned buffers;
``balance_loss`` and ``route_backward`` allocate what is not given.
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import load
from .marshal import DTYPE_CODE, Entry, cuda_device, made, need

_loss = Entry("moe_balance_loss")
_backward = Entry("moe_route_backward")


def moe_balance_workspace_bytes(T: int, E: int, n_seq: int = 1) -> int:
    return int(load().moe_balance_workspace_bytes(T, E, n_seq))


class BalanceBuffers:
    """Outputs and workspace of the balance loss for one (T, E, n_seq): ``loss`` [1] float32,
    ``counts`` [n_seq, E] int32, ``mean_probs`` [n_seq, E] float32.  The buffers are the
    container's own and cannot be exchanged."""

    __slots__ = ("_loss", "_counts", "_mean", "_workspace", "_shape")

    def __init__(self, T: int, E: int, n_seq: int, device):
        ws = moe_balance_workspace_bytes(T, E, n_seq)
        if ws == 0:
            raise ValueError("invalid shape for balance-loss buffers")
        self._loss = torch.empty(1, dtype=torch.float32, device=device)
        self._counts = torch.empty(n_seq, E, dtype=torch.int32, device=device)
        self._mean = torch.empty(n_seq, E, dtype=torch.float32, device=device)
        self._workspace = torch.empty(ws, dtype=torch.uint8, device=device)
        self._shape = (T, E, n_seq, self._loss.get_device())

    loss = property(lambda self: self._loss)
    counts = property(lambda self: self._counts)
    mean_probs = property(lambda self: self._mean)
    workspace = property(lambda self: self._workspace)
    tensors = property(lambda self: (self._loss, self._counts, self._mean, self._workspace))

    @classmethod
    def allocate(cls, T: int, E: int, n_seq: int = 1, device="cuda") -> "BalanceBuffers":
        return cls(T, E, n_seq, device)


def _router(logits, topk_ids, seq_offsets, topk=None):
    """(T, E, K, S, device, addresses of logits, ids, offsets) of a router's call; K is ``topk``
    without ids."""
    dev = cuda_device(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    K, pid = 1 if topk is None else topk, 0
    if topk_ids is not None:
        if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
            raise ValueError("topk_ids must be [T, topk] for logits [T, E]")
        K = topk_ids.shape[1]
        if topk is not None and topk != K:
            raise ValueError(f"topk_ids holds {K} routes per token, topk is {topk}")
        pid = need(topk_ids, torch.int32, 0, dev, "topk_ids")
    S, po = 1, 0
    if seq_offsets is not None:
        S = seq_offsets.numel() - 1
        po = need(seq_offsets, torch.int32, 1, dev, "seq_offsets")
    return T, E, K, S, dev, need(logits, torch.bfloat16, 0, dev, "logits"), pid, po


def moe_balance_loss(logits, topk_ids, seq_offsets: Optional[torch.Tensor], softmax: bool,
                     coef: float, loss, counts, mean_probs, workspace, stream=None) -> None:
    """Balance loss, per-expert counts and mean probabilities into caller-owned buffers.
    ``seq_offsets`` [n_seq + 1] int32, or None for one sequence of all tokens."""
    if topk_ids is None:
        raise ValueError("topk_ids must be [T, topk]")
    T, E, K, S, dev, pl, pid, po = _router(logits, topk_ids, seq_offsets)
    _loss(dev, stream, pl, pid, po, T, E, K, S, 1 if softmax else 0, coef,
          need(loss, torch.float32, 1, dev, "loss"),
          need(counts, torch.int32, S * E, dev, "counts"),
          need(mean_probs, torch.float32, S * E, dev, "mean_probs"),
          need(workspace, torch.uint8, 0, dev, "workspace"), workspace.numel())


def balance_loss(logits, topk_ids, coef: float, softmax: bool = False,
                 seq_offsets: Optional[torch.Tensor] = None,
                 out: Optional[BalanceBuffers] = None, stream=None) -> BalanceBuffers:
    """Allocate (unless ``out`` is given) and run moe_balance_loss; returns the buffers."""
    if topk_ids is None:
        raise ValueError("topk_ids must be [T, topk]")
    T, E, K, S, dev, pl, pid, po = _router(logits, topk_ids, seq_offsets)
    if out is None:
        out = made(dev, stream, lambda: BalanceBuffers.allocate(T, E, S, device=logits.device))
    elif out._shape != (T, E, S, dev):
        raise ValueError(f"out is for (T, E, n_seq, device) {out._shape}, the call is "
                         f"{(T, E, S, dev)}")
    ws = out._workspace
    _loss(dev, stream, pl, pid, po, T, E, K, S, 1 if softmax else 0, coef, out._loss.data_ptr(),
          out._counts.data_ptr(), out._mean.data_ptr(), ws.data_ptr(), ws.numel())
    return out


def moe_route_backward(logits, topk_ids, grad_weights, grad_loss, counts, seq_offsets,
                       softmax: bool, routed_scale: float, coef: float, grad_logits,
                       stream=None, topk: Optional[int] = None) -> None:
    """Gradient to the logits of the routing weights (``grad_weights`` [T, topk], None: no such
    term) and of the balance loss (``grad_loss`` [1] and the ``counts`` of the forward call,
    None: no such term) into ``grad_logits`` [T, E], bfloat16 or float32.  The loss term is
    divided by the routes per token: without ``topk_ids`` (None) it needs ``topk``."""
    T, E, K, S, dev, pl, pid, po = _router(logits, topk_ids, seq_offsets, topk)
    if grad_weights is not None and topk_ids is None:
        raise ValueError("grad_weights needs topk_ids")
    if grad_loss is not None and counts is None:
        raise ValueError("grad_loss needs the counts of the forward call")
    if grad_loss is not None and topk_ids is None and topk is None:
        raise ValueError("grad_loss without topk_ids needs topk, the routes per token")
    dtype = grad_logits.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"grad_logits must be bfloat16 or float32, got {dtype}")
    _backward(dev, stream, pl, pid,
              0 if grad_weights is None else need(grad_weights, torch.float32, T * K, dev,
                                                     "grad_weights"),
              0 if grad_loss is None else need(grad_loss, torch.float32, 1, dev, "grad_loss"),
              0 if counts is None else need(counts, torch.int32, S * E, dev, "counts"),
              po, T, E, K, S, 1 if softmax else 0, routed_scale, coef,
              need(grad_logits, dtype, T * E, dev, "grad_logits"), DTYPE_CODE[dtype])


def route_backward(logits, topk_ids, grad_weights=None, routed_scale: float = 1.0,
                   softmax: bool = False, grad_loss=None, counts=None, coef: float = 0.0,
                   seq_offsets=None, dtype=torch.bfloat16,
                   out: Optional[torch.Tensor] = None, stream=None,
                   topk: Optional[int] = None) -> torch.Tensor:
    """Allocate (unless ``out`` is given) and run moe_route_backward; returns the gradient."""
    if out is None:
        out = made(cuda_device(logits, "logits"), stream,
                   lambda: torch.empty(logits.shape, dtype=dtype, device=logits.device))
    moe_route_backward(logits, topk_ids, grad_weights, grad_loss, counts, seq_offsets, softmax,
                       routed_scale, coef, out, stream, topk)
    return out
