"""Run the route-sort path a fixed number of times on one synthetic workload.

A small driver for external profilers: it builds nothing, allocates the inputs and
outputs of one workload once, issues ``--calls`` back-to-back ``route_sort`` calls on the
current stream and synchronizes.  Example::

    python -m moe_expert_routing_sort_gb300.profile_calls --workload wide_T16384_E4096 --calls 4
    python -m moe_expert_routing_sort_gb300.profile_calls --gate-hidden 7168 --calls 4
    python -m moe_expert_routing_sort_gb300.profile_calls --workload prefill_T512_E896 \
        --operator experts --cols 3584 --outs 768 --calls 3

With ``--operator`` the calls are those of an operator next to the path, on the workload's routes.
"""
from __future__ import annotations

import argparse

import numpy as np


def main(argv=None) -> int:
    from . import datagen

    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--workload", default="decode_T1_E896_G8", choices=list(datagen.WORKLOADS))
    p.add_argument("--calls", type=int, default=8)
    p.add_argument("--tokens", type=int, default=None, help="override the workload's T")
    p.add_argument("--gate-hidden", type=int, default=None,
                   help="run moe_gate_route_sort with this hidden size (gate GEMV ahead)")
    p.add_argument("--operator", choices=("loss", "backward", "quantize", "experts"))
    p.add_argument("--softmax", action="store_true", help="loss and backward of softmax scores")
    p.add_argument("--cols", type=int, default=3584, help="row length of quantize and experts")
    p.add_argument("--outs", type=int, default=768, help="output width of experts")
    args = p.parse_args(argv)

    import torch

    from . import binding

    kw = {} if args.tokens is None else {"T": args.tokens}
    w = datagen.workload(args.workload, **kw)
    inp = datagen.make_inputs(w)
    logits = torch.from_numpy(inp.logits_bf16.view(np.int16)).view(torch.bfloat16).cuda()
    bias = torch.from_numpy(inp.bias).cuda()
    out = binding.RouteSortBuffers.allocate(w.T, w.E, w.topk, w.block_m, device="cuda")
    if args.gate_hidden is not None:
        g = datagen.make_gate_inputs(w.T, w.E, args.gate_hidden, seed=w.seed)
        hid = torch.from_numpy(g.hidden_bf16.view(np.int16)).view(torch.bfloat16).cuda()
        wg = torch.from_numpy(g.w_gate_bf16.view(np.int16)).view(torch.bfloat16).cuda()
        gb = torch.from_numpy(g.bias).cuda()
        for _ in range(args.calls):
            binding.gate_route_sort(hid, wg, gb, w.n_group, w.topk_group, w.topk,
                                    w.routed_scale, w.block_m, out=out, logits=logits)
        torch.cuda.synchronize()
        print(f"{w.name} with gate H={args.gate_hidden}: {args.calls} calls, "
              f"status={out.status_word()}")
        return 0
    if args.operator is not None:
        _operator(args, w, binding.route_sort(logits, bias, w.n_group, w.topk_group, w.topk,
                                              w.routed_scale, w.block_m, out=out), logits)
        print(f"{args.operator} on the routes of {w.name}: {args.calls} calls, T={w.T}")
        return 0
    for _ in range(args.calls):
        binding.route_sort(logits, bias, w.n_group, w.topk_group, w.topk, w.routed_scale,
                           w.block_m, out=out)
    torch.cuda.synchronize()
    print(f"{w.name}: {args.calls} calls, T={w.T}, npp={int(out.num_tokens_post_pad.item())}, "
          f"status={out.status_word()}")
    return 0


def _operator(args, w, r, logits) -> None:
    import torch

    from . import experts, training

    buf = training.BalanceBuffers.allocate(w.T, w.E, 1, device="cuda")
    training.balance_loss(logits, r.topk_ids, 0.01, args.softmax, out=buf)
    grad = torch.empty_like(logits)
    upstream = torch.randn(w.T, w.topk, device="cuda")
    one = torch.ones(1, device="cuda")
    if args.operator in ("quantize", "experts"):
        x = torch.randn(w.T, args.cols, device="cuda").bfloat16()
        rows = experts.mxfp4_quantize(x)
    if args.operator == "experts":
        wts = experts.Mxfp4Rows(
            torch.randint(0, 256, (w.E, args.outs, args.cols // 2), dtype=torch.uint8,
                          device="cuda"),
            torch.randint(120, 128, (w.E, args.outs, rows.scales.shape[1]), dtype=torch.uint8,
                          device="cuda"))
        y = torch.empty(w.routes, args.outs, dtype=torch.bfloat16, device="cuda")
        ws = torch.zeros(experts.moe_experts_mxfp4_workspace_bytes(w.T, w.E, w.topk, w.block_m),
                         dtype=torch.uint8, device="cuda")
    for _ in range(args.calls):
        if args.operator == "loss":
            training.balance_loss(logits, r.topk_ids, 0.01, args.softmax, out=buf)
        elif args.operator == "backward":
            training.route_backward(logits, r.topk_ids, upstream, w.routed_scale, args.softmax,
                                    one, buf.counts, 0.01, out=grad)
        elif args.operator == "quantize":
            experts.mxfp4_quantize(x, out=rows)
        else:
            experts.experts_mxfp4(rows, wts, w.T, w.topk, w.block_m, r.sorted_token_ids,
                                  r.expert_ids, r.num_tokens_post_pad, out=y, workspace=ws)
    torch.cuda.synchronize()


if __name__ == "__main__":
    raise SystemExit(main())
