"""Workloads of the operators that train a router and feed its experts.

Four operators, each next to the route-sort path:

* ``loss``      the balance loss of a router with its per-expert counts and mean probabilities
* ``backward``  the gradient of the routing weights and of that loss to the router logits
* ``quantise``  rows to microscaled 4-bit floating point (blocks of 32, power-of-two scales),
                and back to the values that the codes stand for
* ``experts``   the experts' products of such rows and weights, driven by the sort's metadata

A case is a dict of plain values; ``run`` computes it in elementary torch operations, or with
``own`` set through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32  # elements that share a scale
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the 4-bit codes 0..7


# ------------------------------------------------------------------------------- cases
def _loss(name, T, E, K, S, softmax, tail=0):
    return dict(name=name, op="loss", T=T, E=E, K=K, S=S, softmax=softmax, tail=tail)


def _backward(name, T, E, K, S, softmax, dtype, tail=0):
    return dict(name=name, op="backward", T=T, E=E, K=K, S=S, softmax=softmax, dtype=dtype, tail=tail)


def _quantise(name, rows, cols, dtype):
    return dict(name=name, op="quantise", rows=rows, cols=cols, dtype=dtype)


def _experts(name, T, E, topk, K, N, block_m, per_route, weighted, dtype, skew):
    return dict(name=name, op="experts", T=T, E=E, topk=topk, K=K, N=N, block_m=block_m, per_route=per_route, weighted=weighted, dtype=dtype, skew=skew)


def listed():
    return [
        # a small router's micro-batch: nothing but latency
        _loss("loss T64 E64", 64, 64, 6, 1, False),
        # a packed training batch: ragged sequences, an empty one, padding behind the last
        _loss("loss T8192 E896 packed", 8192, 896, 16, 9, False, tail=77),
        # the largest router, softmax scores, one sequence
        _loss("loss T16384 E4096", 16384, 4096, 8, 1, True),
        # an odd number of experts, gradients in 32 bits for an optimizer that adds them up
        _backward("backward T1000 E129", 1000, 129, 5, 3, True, "float32"),
        # the backward pass of the packed training batch
        _backward("backward T8192 E896 packed", 8192, 896, 16, 9, False, "bfloat16", tail=77),
        # one token's sixteen intermediate rows between the two products: latency
        _quantise("quantise 16x384", 16, 384, "bfloat16"),
        # a prefill's latent rows ahead of the first product
        _quantise("quantise 8192x3584", 8192, 3584, "bfloat16"),
        # one decoded token through the first product: sixteen experts' weights are read once
        _experts("experts up T1", 1, 896, 16, 3584, 768, 16, False, False, "bfloat16", False),
        # and through the second, weighted, in 32 bits for the sum over its experts
        _experts("experts down T1", 1, 896, 16, 384, 3584, 16, True, True, "float32", False),
        # a prefill of 512 tokens: about nine rows an expert, nearly every expert's weights
        _experts("experts up T512", 512, 896, 16, 3584, 768, 32, False, False, "bfloat16", False),
        # a long prefill whose router prefers some experts, second product
        _experts("experts down T8192 skewed", 8192, 896, 16, 384, 3584, 128, True, True, "bfloat16", True),
        # few experts with wide layers: a thousand rows each, bound by arithmetic
        _experts("experts up T8192 E64", 8192, 64, 8, 7168, 2048, 128, False, False, "bfloat16", False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["loss", "backward", "quantise", "experts", "experts"])
    if op in ("loss", "backward"):
        E = _log_int(rng, 8, 4096)
        if rng.random() < 0.5:
            E = max(8, E // 8 * 8)
        T = _log_int(rng, 1, min(16384, 16384 * 4096 // E))
        K = rng.randint(1, min(32, E))
        S = rng.choice([1, rng.randint(1, 40)])
        c = dict(op=op, T=T, E=E, K=K, S=S, softmax=rng.random() < 0.5, tail=rng.choice([0, rng.randint(0, T // 4)]))
        if op == "backward":
            c["dtype"] = rng.choice(["bfloat16", "float32"])
        return c
    if op == "quantise":
        rows = _log_int(rng, 1, 40000)
        cols = BLOCK * _log_int(rng, 1, max(1, min(512, 8192 * 3584 // (rows * BLOCK))))
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bfloat16", "float16", "float32"]))
    while True:
        E, T = _log_int(rng, 4, 896), _log_int(rng, 1, 8192)
        topk = rng.randint(1, min(16, E))
        K, N = BLOCK * _log_int(rng, 2, 224), 8 * _log_int(rng, 8, 448)
        block_m = rng.choice([8, 16, 32, 64, 128, 256])
        rows = T * topk + min(E, T * topk) * (block_m - 1)
        blocks = rows // block_m
        if max(blocks, 1) * N * K > 5e9 or E * N * K > 2e9 or rows * (N + K) > 2e9 or 2.0 * rows * N * K > 2e12:
            continue
        return dict(op=op, T=T, E=E, topk=topk, K=K, N=N, block_m=block_m, per_route=rng.random() < 0.5, weighted=rng.random() < 0.5,
                    dtype=rng.choice(["bfloat16", "float32"]), skew=rng.random() < 0.5)


# ------------------------------------------------------------------------------ inputs
def _choose(g, T, E, K, skew):
    """K different experts for each token, best first, and the logits they come from."""
    x = torch.randn(T, E, generator=g, device=DEV)
    if skew:  # a few hot experts, by a power law of their rank
        rank = 1.0 + torch.randperm(E, generator=g, device=DEV).float()
        x = x - 0.55 * rank.log()
    x = x.bfloat16()
    return x, x.float().topk(K, dim=1).indices.int()


def _prepare_router(c, g):
    T, E, K, S = c["T"], c["E"], c["K"], c["S"]
    logits, ids = _choose(g, T, E, K, True)
    # S sequences one behind another (two equal borders: an empty one), padding behind the last
    end = T - c["tail"]
    cuts = torch.randint(0, end + 1, (S - 1,), generator=g, device=DEV).sort().values
    offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), end)]).int()
    if S >= 9:
        offsets[4] = offsets[5]
    ids[end:] = -1  # the padding's routes are dropped
    s = dict(c, logits=logits, ids=ids.contiguous(), offsets=offsets, coef=0.01, scale=2.5, kept={})
    if c["op"] == "backward":
        s["grad_weights"] = torch.randn(T, K, generator=g, device=DEV) / T
        s["grad_loss"] = torch.rand(1, generator=g, device=DEV) + 0.5
        s["counts"] = _counts(ids, offsets, E)
    return s


def _sort_rows(ids, weights, E, B):
    """The sort step's metadata for these routes: rows grouped by expert, padded to blocks."""
    flat, n = ids.reshape(-1).long(), ids.numel()
    count = torch.bincount(flat, minlength=E)
    pad = (count + B - 1) // B * B
    last = pad.cumsum(0)
    order = flat.argsort(stable=True)
    e = flat[order]
    place = (last - pad)[e] + torch.arange(n, device=DEV) - (count.cumsum(0) - count)[e]
    P = n + min(n, E) * (B - 1)
    sid = torch.full((P,), n, dtype=torch.int32, device=DEV)
    sw = torch.zeros(P, device=DEV)
    sid[place] = order.int()
    sw[place] = weights.reshape(-1)[order]
    eid = torch.bucketize(torch.arange(P // B, device=DEV) * B, last, right=True).clamp_(max=E - 1).int()
    return sid, sw, eid, last[-1:].int()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] in ("loss", "backward"):
        return _prepare_router(c, g)
    if c["op"] == "quantise":
        # activations: rows of different size, a few columns that stand out
        x = torch.randn(c["rows"], c["cols"], generator=g, device=DEV)
        x *= torch.exp(torch.randn(c["rows"], 1, generator=g, device=DEV))
        x *= 1.0 + 20.0 * (torch.rand(1, c["cols"], generator=g, device=DEV) < 0.01).float()
        return dict(c, x=x.to(getattr(torch, c["dtype"])), kept={})
    T, E, topk, K, N = c["T"], c["E"], c["topk"], c["K"], c["N"]
    _, ids = _choose(g, T, E, topk, c["skew"])
    weights = torch.rand(T, topk, generator=g, device=DEV) + 0.1
    weights = 2.5 * weights / weights.sum(1, keepdim=True)
    sid, sw, eid, npp = _sort_rows(ids, weights, E, c["block_m"])
    xc, xs = _quantise_plain(torch.randn(T * topk if c["per_route"] else T, K, generator=g, device=DEV))
    wc = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    ws = torch.randint(118, 123, (E, N, xs.shape[1]), generator=g, device=DEV, dtype=torch.uint8)
    ws[:, :, K // BLOCK:] = 0
    return dict(c, xc=xc, xs=xs, wc=wc, ws=ws, sid=sid, sw=sw, eid=eid, npp=npp, kept={})


# ------------------------------------------------------------------------- plain forms
def _sequence_of(offsets, T):
    """The sequence of each token; S for a token that belongs to none."""
    S = offsets.numel() - 1
    q = torch.bucketize(torch.arange(T, device=offsets.device, dtype=torch.int32), offsets, right=True) - 1
    return torch.where((q >= 0) & (q < S), q, S).long()


def _counts(ids, offsets, E):
    q, S = _sequence_of(offsets, ids.shape[0]), offsets.numel() - 1
    fine = (ids >= 0) & (ids < E)
    at = torch.where(fine, q[:, None] * E + ids.long(), S * E)
    return torch.bincount(at.reshape(-1), minlength=(S + 1) * E)[: S * E].reshape(S, E).int()


def _probabilities(x, softmax):
    if softmax:
        e = (x - x.amax(1, keepdim=True)).exp()
        return e / e.sum(1, keepdim=True), None
    s = 1.0 / (1.0 + (-x).exp())
    return s / s.sum(1, keepdim=True), s


def _loss_plain(s):
    E, S = s["E"], s["S"]
    p, _ = _probabilities(s["logits"].float(), s["softmax"])
    q = _sequence_of(s["offsets"], s["T"])
    total = torch.zeros(S + 1, E, dtype=torch.float64, device=DEV).index_add_(0, q, p.double())[:S]
    n = s["offsets"].diff().double().clamp(min=1)[:, None]
    counts = _counts(s["ids"], s["offsets"], E)
    mean = total / n
    loss = s["coef"] / S * (counts.double() * (E / s["K"]) / n * mean).sum()
    return {"loss": loss.float().reshape(1), "counts": counts, "mean_probs": mean.float()}


def _backward_plain(s):
    T, E, K, S = s["T"], s["E"], s["K"], s["S"]
    x = s["logits"].float()
    p, sig = _probabilities(x, s["softmax"])
    q = _sequence_of(s["offsets"], T)
    n = s["offsets"].diff().float().clamp(min=1)[:, None]
    g = s["grad_loss"] * (s["coef"] / S) * (E / K) * s["counts"].float() / (n * n)
    g = torch.cat([g, g.new_zeros(1, E)])[q]
    d = g - (p * g).sum(1, keepdim=True)
    d = d * p if s["softmax"] else d * p * (1.0 - sig)
    # the weights: w_k = scale * u_k / sum u over the token's valid routes
    ids, gw = s["ids"], s["grad_weights"]
    fine = (ids >= 0) & (ids < E)
    at = torch.where(fine, ids, 0).long()
    xk = x.gather(1, at).masked_fill(~fine, -math.inf)
    top = xk.amax(1, keepdim=True).clamp(min=-3e38)
    u = (xk - top).exp() if s["softmax"] else 1.0 / (1.0 + (-xk).exp())
    share = u / u.sum(1, keepdim=True).clamp(min=1e-30)
    gw = torch.where(fine, gw, 0.0)
    dk = s["scale"] * share * (gw - (share * gw).sum(1, keepdim=True))
    if not s["softmax"]:
        dk = dk * (1.0 - u)
    return d.scatter_add_(1, at, torch.where(fine, dk, 0.0)).to(getattr(torch, s["dtype"]))


def _quantise_plain(x):
    rows, cols = x.shape
    b = x.float().reshape(rows, cols // BLOCK, BLOCK)
    # the shared exponent: that of the largest magnitude, less the 2 of the largest code
    e = (torch.frexp(b.abs().amax(2)).exponent - 3).clamp(-127, 125)
    e = torch.where(b.abs().amax(2) > 0, e, -127)
    a = b * ((127 - e) << 23).view(torch.float32)[:, :, None]  # 2^-e from its bits
    m = a.abs()
    # nearest of the grid, ties to the even code, the largest code for all beyond
    code = (m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    code = (code + 8 * torch.signbit(a)).byte().reshape(rows, cols)
    scales = torch.zeros(rows, (cols + 127) // 128 * 4, dtype=torch.uint8, device=x.device)
    scales[:, : cols // BLOCK] = (e + 127).byte()
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def _values(codes, scales):
    """What codes [..., cols / 2] and scales [..., at least cols / 32] stand for, in 32 bits."""
    one = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)  # of each byte: low, high
    v = pair[codes.int()].reshape(*codes.shape[:-1], -1, BLOCK)
    e = scales[..., : v.shape[-2]].int()
    step = torch.where(e > 0, e << 23, 1 << 22).view(torch.float32)  # 2^(e - 127) from its bits
    return v.mul_(step[..., None]).flatten(-2)


def _experts_plain(s):
    T, topk, B, N = s["T"], s["topk"], s["block_m"], s["N"]
    n, blocks = T * topk, s["eid"].numel()
    sid = s["sid"][: blocks * B].long()
    row = (sid if s["per_route"] else sid // topk).clamp(max=s["xc"].shape[0] - 1)
    x = _values(s["xc"], s["xs"])[row].reshape(blocks, B, -1)
    w = _values(s["wc"], s["ws"])[s["eid"].long()]
    y = torch.bmm(x, w.transpose(1, 2)).reshape(blocks * B, N)
    if s["weighted"]:
        y = y * s["sw"][: blocks * B, None]
    out = torch.zeros(n + 1, N, device=DEV).index_copy_(0, sid, y)  # padding rows: the last
    return out[:n].to(getattr(torch, s["dtype"]))


# -------------------------------------------------------------------- the package's calls
def _own(s):
    import moe_expert_routing_sort_gb300 as mrs

    kept = s["kept"]
    if s["op"] == "loss":
        if not kept:
            kept["out"] = mrs.BalanceBuffers.allocate(s["T"], s["E"], s["S"], device=DEV)
        out = mrs.balance_loss(s["logits"], s["ids"], s["coef"], softmax=s["softmax"], seq_offsets=s["offsets"], out=kept["out"])
        return {"loss": out.loss, "counts": out.counts, "mean_probs": out.mean_probs}
    if s["op"] == "backward":
        if not kept:
            kept["grad"] = torch.empty(s["T"], s["E"], dtype=getattr(torch, s["dtype"]), device=DEV)
        return mrs.route_backward(s["logits"], s["ids"], grad_weights=s["grad_weights"], routed_scale=s["scale"], softmax=s["softmax"],
                                  grad_loss=s["grad_loss"], counts=s["counts"], coef=s["coef"], seq_offsets=s["offsets"], out=kept["grad"])
    if s["op"] == "quantise":
        if not kept:
            kept["rows"] = mrs.Mxfp4Rows.allocate(s["rows"], s["cols"], device=DEV)
            kept["values"] = torch.empty(s["rows"], s["cols"], dtype=torch.bfloat16, device=DEV)
        return mrs.mxfp4_dequantize(mrs.mxfp4_quantize(s["x"], out=kept["rows"]), out=kept["values"])
    if not kept:
        kept["x"] = mrs.Mxfp4Rows(s["xc"], s["xs"])
        kept["w"] = mrs.Mxfp4Rows(s["wc"], s["ws"])
        kept["out"] = torch.empty(s["T"] * s["topk"], s["N"], dtype=getattr(torch, s["dtype"]), device=DEV)
        kept["ws"] = torch.zeros(mrs.moe_experts_mxfp4_workspace_bytes(s["T"], s["E"], s["topk"], s["block_m"]), dtype=torch.uint8, device=DEV)
    return mrs.experts_mxfp4(kept["x"], kept["w"], s["T"], s["topk"], s["block_m"], s["sid"], s["eid"], s["npp"],
                             sorted_weights=s["sw"] if s["weighted"] else None, out=kept["out"], workspace=kept["ws"])


def run(state):
    if own:
        return _own(state)
    if state["op"] == "loss":
        return _loss_plain(state)
    if state["op"] == "backward":
        return _backward_plain(state)
    if state["op"] == "quantise":
        return _values(*_quantise_plain(state["x"])).bfloat16()
    return _experts_plain(state)


# ------------------------------------------------------------------------- what it takes
def work(case):
    c = case
    if c["op"] in ("loss", "backward"):
        T, E, K, S = c["T"], c["E"], c["K"], c["S"]
        if c["op"] == "loss":
            return {"bytes": 2 * T * E + 4 * T * K + 8 * S * E, "flops": 6 * T * E}
        size = 4 if c["dtype"] == "float32" else 2
        return {"bytes": (2 + size) * T * E + 8 * T * K + 4 * S * E, "flops": 10 * T * E}
    if c["op"] == "quantise":
        n = c["rows"] * c["cols"]
        size = 4 if c["dtype"] == "float32" else 2
        # the input, the codes and scales written and read again, the values
        return {"bytes": n * size + 2 * (n // 2 + n // BLOCK) + 2 * n, "flops": 4 * n}
    T, E, topk, K, N = c["T"], c["E"], c["topk"], c["K"], c["N"]
    hit = min(float(T * topk), E * (1.0 - (1.0 - topk / E) ** T))  # experts with any row
    row = K / 2 + K / BLOCK
    size = 4 if c["dtype"] == "float32" else 2
    return {"bytes": hit * N * row + (T * topk if c["per_route"] else T) * row + T * topk * (N * size + 4), "flops": 2.0 * T * topk * N * K}


# ------------------------------------------------------- from the definitions, in 64 bits
def _exact_loss(logits, ids, offsets, E, K, coef, softmax):
    S, loss, counts, means = len(offsets) - 1, 0.0, [], []
    for a, b in zip(offsets[:-1], offsets[1:]):
        x, i = logits[a:b], ids[a:b].reshape(-1).long()
        count = torch.bincount(i[(i >= 0) & (i < E)], minlength=E)
        p = torch.softmax(x, 1) if softmax else torch.sigmoid(x) / torch.sigmoid(x).sum(1, keepdim=True)
        mean = p.sum(0) / max(b - a, 1)
        loss = loss + coef / S * (count.double() * E / (K * max(b - a, 1))).dot(mean)
        counts.append(count)
        means.append(mean)
    return loss, torch.stack(counts), torch.stack(means)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "loss":
        loss, counts, means = _exact_loss(s["logits"].double(), s["ids"], s["offsets"].tolist(), s["E"], s["K"], s["coef"], s["softmax"])
        return {"loss": loss.reshape(1), "counts": counts.int(), "mean_probs": means}
    if s["op"] == "backward":  # by differentiating the definitions
        x = s["logits"].double().requires_grad_()
        loss, _, _ = _exact_loss(x, s["ids"], s["offsets"].tolist(), s["E"], s["K"], s["coef"], s["softmax"])
        fine = (s["ids"] >= 0).double()
        score = torch.exp(x - x.detach().amax(1, keepdim=True)) if s["softmax"] else torch.sigmoid(x)
        u = score.gather(1, s["ids"].clamp(min=0).long()) * fine
        w = s["scale"] * u / (u.sum(1, keepdim=True) + (1.0 - fine).prod(1, keepdim=True))
        total = loss * s["grad_loss"].double() + (w * s["grad_weights"].double()).sum()
        return torch.autograd.grad(total.sum(), x)[0]
    if s["op"] == "quantise":
        b = s["x"].double().unflatten(1, (-1, BLOCK))
        top = b.abs().amax(2, keepdim=True)
        e = torch.floor(torch.log2(top.clamp(min=1e-60))).long()
        power = lambda k: ((k + 1023) << 52).view(torch.float64)  # noqa: E731
        e = e + (power(e + 1) <= top).long() - (power(e) > top).long()  # log2 may be off by its last place
        step = power((e - 2).clamp(-127, 125))
        v, grid = (b / step).abs(), torch.tensor(GRID, dtype=torch.float64, device=DEV)
        low = torch.searchsorted(grid, v.contiguous(), right=True).clamp(1, 7) - 1
        to_low, to_high = v - grid[low], grid[low + 1] - v
        up = (to_high < to_low) | ((to_high == to_low) & (low % 2 == 1))
        return (torch.where(b < 0, -1.0, 1.0) * grid[low + up] * step).flatten(1)
    T, topk, B, N, K = s["T"], s["topk"], s["block_m"], s["N"], s["K"]
    if 2.0 * s["sid"].numel() * N * K > 8e12:
        return None
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=DEV)

    def value(codes, scales):
        v = grid[torch.stack([codes & 15, codes >> 4], -1).long()].flatten(-2).unflatten(-1, (-1, BLOCK))
        return (v * ((scales[..., : K // BLOCK].long() + (1023 - 127)) << 52).view(torch.float64)[..., None]).flatten(-2)

    out = torch.zeros(T * topk, N, dtype=torch.float64, device=DEV)
    x = value(s["xc"], s["xs"])
    used = int(s["npp"]) // B
    owner = s["eid"][:used].repeat_interleave(B)
    sid, sw = s["sid"][: used * B].long(), s["sw"][: used * B].double()
    for e in s["eid"][:used].unique().tolist():
        at = ((owner == e) & (sid < T * topk)).nonzero()[:, 0]
        r = sid[at]
        y = x[r if s["per_route"] else r // topk] @ value(s["wc"][e], s["ws"][e]).T
        out[r] = y * sw[at, None] if s["weighted"] else y
    return out
