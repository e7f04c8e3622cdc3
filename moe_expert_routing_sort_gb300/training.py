"""Training a router: its balance loss with per-expert counts, and the gradient of the routing
weights and of that loss to the logits (see include/moe_route_sort.h).

``moe_*`` functions have the names of their C entry points and fill caller-owned buffers;
``balance_loss`` and ``route_backward`` allocate what is not given.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from .binding import load
from .marshal import DTYPE_CODE, cuda_device, launch, need


def moe_balance_workspace_bytes(T: int, E: int, n_seq: int = 1) -> int:
    return int(load().moe_balance_workspace_bytes(T, E, n_seq))


@dataclass
class BalanceBuffers:
    """Outputs and workspace of the balance loss for one (T, E, n_seq)."""

    loss: torch.Tensor        # [1] float32
    counts: torch.Tensor      # [n_seq, E] int32
    mean_probs: torch.Tensor  # [n_seq, E] float32
    workspace: torch.Tensor

    @classmethod
    def allocate(cls, T: int, E: int, n_seq: int = 1, device="cuda") -> "BalanceBuffers":
        ws = moe_balance_workspace_bytes(T, E, n_seq)
        if ws == 0:
            raise ValueError("invalid shape for balance-loss buffers")
        return cls(torch.empty(1, dtype=torch.float32, device=device),
                   torch.empty(n_seq, E, dtype=torch.int32, device=device),
                   torch.empty(n_seq, E, dtype=torch.float32, device=device),
                   torch.empty(ws, dtype=torch.uint8, device=device))


def _router(logits, topk_ids, seq_offsets):
    """(T, E, K, S, device, addresses of logits, ids, offsets) of a router's call."""
    dev = cuda_device(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    K, pid = 1, None
    if topk_ids is not None:
        if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
            raise ValueError("topk_ids must be [T, topk] for logits [T, E]")
        K = topk_ids.shape[1]
        pid = need(topk_ids, torch.int32, T * K, dev, "topk_ids")
    S, po = 1, None
    if seq_offsets is not None:
        S = seq_offsets.numel() - 1
        po = need(seq_offsets, torch.int32, 1, dev, "seq_offsets")
    return T, E, K, S, dev, need(logits, torch.bfloat16, T * E, dev, "logits"), pid, po


def moe_balance_loss(logits, topk_ids, seq_offsets: Optional[torch.Tensor], softmax: bool,
                     coef: float, loss, counts, mean_probs, workspace, stream=None) -> None:
    """Balance loss, per-expert counts and mean probabilities into caller-owned buffers.
    ``seq_offsets`` [n_seq + 1] int32, or None for one sequence of all tokens."""
    if topk_ids is None:
        raise ValueError("topk_ids must be [T, topk]")
    T, E, K, S, dev, pl, pid, po = _router(logits, topk_ids, seq_offsets)
    launch("moe_balance_loss", dev, stream, pl, pid, po, T, E, K, S, int(softmax), float(coef),
           need(loss, torch.float32, 1, dev, "loss"),
           need(counts, torch.int32, S * E, dev, "counts"),
           need(mean_probs, torch.float32, S * E, dev, "mean_probs"),
           need(workspace, torch.uint8, 0, dev, "workspace"), workspace.numel())


def balance_loss(logits, topk_ids, coef: float, softmax: bool = False,
                 seq_offsets: Optional[torch.Tensor] = None,
                 out: Optional[BalanceBuffers] = None, stream=None) -> BalanceBuffers:
    """Allocate (unless ``out`` is given) and run moe_balance_loss; returns the buffers."""
    if out is None:
        S = 1 if seq_offsets is None else seq_offsets.numel() - 1
        out = BalanceBuffers.allocate(logits.shape[0], logits.shape[1], S, device=logits.device)
    moe_balance_loss(logits, topk_ids, seq_offsets, softmax, coef, out.loss, out.counts,
                     out.mean_probs, out.workspace, stream=stream)
    return out


def moe_route_backward(logits, topk_ids, grad_weights, grad_loss, counts, seq_offsets,
                       softmax: bool, routed_scale: float, coef: float, grad_logits,
                       stream=None) -> None:
    """Gradient to the logits of the routing weights (``grad_weights`` [T, topk], None: no such
    term) and of the balance loss (``grad_loss`` [1] and the ``counts`` of the forward call,
    None: no such term) into ``grad_logits`` [T, E], bfloat16 or float32."""
    T, E, K, S, dev, pl, pid, po = _router(logits, topk_ids, seq_offsets)
    if grad_weights is not None and topk_ids is None:
        raise ValueError("grad_weights needs topk_ids")
    if grad_loss is not None and counts is None:
        raise ValueError("grad_loss needs the counts of the forward call")
    if grad_logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"grad_logits must be bfloat16 or float32, got {grad_logits.dtype}")
    pw = None if grad_weights is None else need(grad_weights, torch.float32, T * K, dev,
                                                "grad_weights")
    pg = None if grad_loss is None else need(grad_loss, torch.float32, 1, dev, "grad_loss")
    pc = None if counts is None else need(counts, torch.int32, S * E, dev, "counts")
    launch("moe_route_backward", dev, stream, pl, pid, pw, pg, pc, po, T, E, K, S, int(softmax),
           float(routed_scale), float(coef),
           need(grad_logits, grad_logits.dtype, T * E, dev, "grad_logits"),
           DTYPE_CODE[grad_logits.dtype])


def route_backward(logits, topk_ids, grad_weights=None, routed_scale: float = 1.0,
                   softmax: bool = False, grad_loss=None, counts=None, coef: float = 0.0,
                   seq_offsets=None, dtype=torch.bfloat16,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Allocate (unless ``out`` is given) and run moe_route_backward; returns the gradient."""
    if out is None:
        out = torch.empty(logits.shape, dtype=dtype, device=logits.device)
    moe_route_backward(logits, topk_ids, grad_weights, grad_loss, counts, seq_offsets, softmax,
                       routed_scale, coef, out, stream=stream)
    return out
