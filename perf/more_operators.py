"""Workloads of the operators between two routings: norm, experts' products, gated activation.

Three operators next to the route-sort path, in each direction that they have:

* ``norm``     root-mean-square norm of the residual plus the sum of a token's expert rows, with an
               8-bit output (e4m3 and a scale for each row), and its gradient
* ``gated``    the gated activation between two experts' products, times the routing weight, and
               its gradient, that of the routing weights included
* ``experts``  the experts' products in 16 or 8 bits, driven by the sort's metadata, and the
               gradients of their rows and of their weights

A case is a dict of plain values; ``run`` computes it in elementary torch operations, or with
``own`` set through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TOP = 448.0  # the largest e4m3 value
TINY = 2.0 ** -126  # the smallest scale


# ------------------------------------------------------------------------------- cases
def _norm(name, T, cols, parts, backward, fp8, dtype):
    return dict(name=name, op="norm", T=T, cols=cols, parts=parts, backward=backward, fp8=fp8, dtype=dtype)


def _gated(name, rows, cols, backward, weighted, fp8, dtype):
    return dict(name=name, op="gated", rows=rows, cols=cols, backward=backward, weighted=weighted, fp8=fp8, dtype=dtype)


def _experts(name, T, E, topk, K, N, block_m, per_route, backward, weighted, dtype, out, skew, drop=False):
    return dict(name=name, op="experts", T=T, E=E, topk=topk, K=K, N=N, block_m=block_m, per_route=per_route, backward=backward,
                weighted=weighted, dtype=dtype, out=out, skew=skew, drop=drop)


def listed():
    return [
        # one decoded token: its sixteen experts' rows onto the residual, normed for the next layer: latency
        _norm("norm T1 3584 of 16", 1, 3584, 16, False, True, "bfloat16"),
        # a prefill ahead of 8-bit products, one row a token
        _norm("norm T8192 3584 fp16", 8192, 3584, 1, False, True, "float16"),
        # the gradient behind a layer of eight experts a token
        _norm("norm backward T8192 7168 of 8", 8192, 7168, 8, True, False, "bfloat16"),
        # one decoded token's sixteen intermediate rows, to 8 bits: latency
        _gated("gated 16x384", 16, 384, False, False, True, "bfloat16"),
        # a training batch of many narrow experts, with the routing weights
        _gated("gated 131072x384", 131072, 384, False, True, False, "bfloat16"),
        # the gradient of a batch of few wide experts, the routing weights' included
        _gated("gated backward 65536x2048", 65536, 2048, True, True, False, "bfloat16"),
        # one decoded token through the first product in 8 bits: sixteen experts' weights are read once
        _experts("experts up T1 fp8", 1, 896, 16, 3584, 768, 16, False, False, False, "float8_e4m3fn", "bfloat16", False),
        # a prefill of 512 tokens: about nine rows an expert, nearly every expert's weights
        _experts("experts up T512", 512, 896, 16, 3584, 768, 32, False, False, False, "bfloat16", "bfloat16", False),
        # few experts with wide layers: a thousand rows each, bound by arithmetic
        _experts("experts up T8192 E64", 8192, 64, 8, 7168, 2048, 128, False, False, False, "bfloat16", "bfloat16", False),
        # a long prefill whose router prefers some experts, second product in 8 bits, weighted
        _experts("experts down T8192 skewed fp8", 8192, 896, 16, 384, 3584, 64, True, False, True, "float8_e4m3fn", "bfloat16", True),
        # an odd number of experts and ragged groups, some routes dropped, 16-bit weight gradients
        _experts("experts backward T1000 E129 fp16", 1000, 129, 6, 520, 264, 16, True, True, False, "float16", "float16", True, drop=True),
        # the training step of few wide experts, weight gradients in 32 bits for an optimizer that adds them up
        _experts("experts backward T8192 E64", 8192, 64, 8, 7168, 2048, 128, False, True, False, "bfloat16", "float32", False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gated", "experts", "experts"])
    half = rng.choice(["bfloat16", "float16"])
    backward = rng.random() < 0.5
    if op == "norm":
        cols, parts = 8 * _log_int(rng, 8, 1024), rng.randint(1, 16)
        T = _log_int(rng, 1, max(1, min(16384, 8192 * 7168 * 9 // (cols * (parts + 1)))))
        return dict(op=op, T=T, cols=cols, parts=parts, backward=backward, fp8=not backward and rng.random() < 0.5, dtype=half)
    if op == "gated":
        cols = 8 * _log_int(rng, 4, 512)
        rows = _log_int(rng, 1, max(1, 65536 * 2048 // cols))
        return dict(op=op, rows=rows, cols=cols, backward=backward, weighted=rng.random() < 0.5, fp8=not backward and rng.random() < 0.5, dtype=half)
    while True:
        E, T = _log_int(rng, 4, 896), _log_int(rng, 1, 8192)
        topk = rng.randint(1, min(16, E))
        eight = not backward and rng.random() < 0.4
        K, N = 16 * _log_int(rng, 4, 448), 8 * _log_int(rng, 8, 448)
        block_m = rng.choice([16, 32, 64, 128])
        rows = T * topk + min(E, T * topk) * (block_m - 1)
        blocks = rows // block_m
        if max(blocks, 1) * N * K > 8e9 or E * N * K > 2e9 or rows * (N + K) > 2e9 or 2.0 * rows * N * K > 2e12:
            continue
        out = rng.choice(["float32", "bfloat16" if eight else half])
        return dict(op=op, T=T, E=E, topk=topk, K=K, N=N, block_m=block_m, per_route=rng.random() < 0.5, backward=backward,
                    weighted=not backward and rng.random() < 0.5, dtype="float8_e4m3fn" if eight else half, out=out, skew=rng.random() < 0.5,
                    drop=rng.random() < 0.3)


# ------------------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _activations(g, rows, cols):
    """Rows of different size, a few columns that stand out."""
    x = _randn(g, rows, cols)
    x *= torch.exp(0.5 * _randn(g, rows, 1))
    x *= 1.0 + 10.0 * (torch.rand(1, cols, generator=g, device=DEV) < 0.01).float()
    return x


def _prepare_norm(c, g):
    T, cols, parts, dtype = c["T"], c["cols"], c["parts"], getattr(torch, c["dtype"])
    gain = (1.0 + 0.2 * _randn(g, cols)).to(dtype)
    residual = _activations(g, T, cols).to(dtype)
    rows = (0.3 * _randn(g, T * parts, cols)).to(dtype)
    if not c["backward"]:
        return dict(c, x=rows, residual=residual, gain=gain, kept={})
    # what a training step kept of the forward call, and the gradients that reach it: one row of
    # each of the token's experts, the router's row, and that of the residual stream
    rstd = (residual.float().square().mean(1) + EPS).rsqrt()
    return dict(c, s=residual, rstd=rstd, gain=gain, grad_rows=rows, grad=_randn(g, T, cols).to(dtype), grad_sum=_randn(g, T, cols).to(dtype), kept={})


def _prepare_gated(c, g):
    rows, cols, dtype = c["rows"], c["cols"], getattr(torch, c["dtype"])
    s = dict(c, x=(2.0 * _randn(g, rows, 2 * cols)).to(dtype), weights=None, kept={})
    if c["weighted"]:
        s["weights"] = torch.rand(rows, generator=g, device=DEV) + 0.05
    if c["backward"]:
        s["grad"] = _randn(g, rows, cols).to(dtype)
    return s


def _sort_rows(ids, weights, E, B):
    """The sort step's metadata for these routes: rows grouped by expert, padded to blocks;
    negative ids are dropped routes."""
    flat, n = ids.reshape(-1).long(), ids.numel()
    key = torch.where(flat < 0, E, flat)
    count = torch.bincount(key, minlength=E + 1)[:E]
    pad = (count + B - 1) // B * B
    last = pad.cumsum(0)
    order = key.argsort(stable=True)
    e = key[order]
    P = n + min(n, E) * (B - 1)
    start, before = torch.cat([last - pad, last.new_full((1,), P)]), torch.cat([count.cumsum(0) - count, count.sum()[None]])
    place = (start[e] + torch.arange(n, device=DEV) - before[e]).clamp(max=P)  # dropped ones: behind the list
    sid = torch.full((P + 1,), n, dtype=torch.int32, device=DEV)
    sw = torch.zeros(P + 1, device=DEV)
    sid[place] = order.int()
    sw[place] = weights.reshape(-1)[order]
    eid = torch.bucketize(torch.arange(P // B, device=DEV) * B, last, right=True).clamp_(max=E - 1).int()
    sid[P] = n
    return sid[:P].contiguous(), sw[:P].contiguous(), eid, last[-1:].int()


def _rows8(x):
    """e4m3 rows with a scale for each, and the scales."""
    scale = (x.abs().amax(-1) / TOP).clamp(min=TINY)
    return (x / scale[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "norm":
        return _prepare_norm(c, g)
    if c["op"] == "gated":
        return _prepare_gated(c, g)
    T, E, topk, K, N = c["T"], c["E"], c["topk"], c["K"], c["N"]
    logits = _randn(g, T, E)
    if c["skew"]:  # a few hot experts, by a power law of their rank
        logits -= 0.55 * (1.0 + torch.randperm(E, generator=g, device=DEV).float()).log()
    ids = logits.topk(topk, dim=1).indices.int()
    if c["drop"]:
        ids = torch.where(torch.rand(T, topk, generator=g, device=DEV) < 0.1, -1, ids)
    weights = torch.rand(T, topk, generator=g, device=DEV) + 0.1
    weights = 2.5 * weights / weights.sum(1, keepdim=True)
    sid, sw, eid, npp = _sort_rows(ids, weights, E, c["block_m"])
    s = dict(c, sid=sid, sw=sw, eid=eid, npp=npp, xs=None, ws=None, kept={})
    x = _randn(g, T * topk if c["per_route"] else T, K)
    if c["dtype"] == "float8_e4m3fn":
        s["x"], s["xs"] = _rows8(x)
        s["w"] = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=DEV)
        s["w"].copy_(_randn(g, E, N, K).mul_(100.0).clamp_(-TOP, TOP))
        s["ws"] = torch.exp(0.3 * _randn(g, E, N)) * (0.01 / math.sqrt(K))
        return s
    dtype = getattr(torch, c["dtype"])
    s["x"] = x.to(dtype)
    s["w"] = torch.empty(E, N, K, dtype=dtype, device=DEV)
    s["w"].copy_(_randn(g, E, N, K).mul_(1.0 / math.sqrt(K)))
    if c["backward"]:  # the gradient of the product's rows, one for each route
        s["grad"] = _randn(g, T * topk, N).to(dtype)
    return s


# ------------------------------------------------------------------------- plain forms
def _norm_plain(s):
    T, cols, parts, dtype = s["T"], s["cols"], s["parts"], getattr(torch, s["dtype"])
    gain = s["gain"].float()
    if not s["backward"]:
        total = (s["residual"].float() + s["x"].float().reshape(T, parts, cols).sum(1)).to(dtype)
        t = total.float()  # the norm is that of the stored sum
        y = t * (t.square().mean(1, keepdim=True) + EPS).rsqrt() * gain
        if not s["fp8"]:
            return {"y": y.to(dtype), "sum": total}
        codes, scales = _rows8(y)
        return {"y": y.to(dtype), "sum": total, "codes": codes, "scales": scales}
    d = s["grad"].float() + s["grad_rows"].float().reshape(T, parts, cols).sum(1)
    xh = s["s"].float() * s["rstd"][:, None]
    dg = d * gain
    dx = s["rstd"][:, None] * (dg - xh * (dg * xh).mean(1, keepdim=True)) + s["grad_sum"].float()
    return {"grad_x": dx.to(dtype), "grad_gain": (d * xh).double().sum(0).float()}


def _gated_plain(s):
    cols, dtype = s["cols"], getattr(torch, s["dtype"])
    x = s["x"].float()
    a, b = x[:, :cols], x[:, cols:]
    w = 1.0 if s["weights"] is None else s["weights"][:, None]
    sig = 1.0 / (1.0 + (-a).exp())
    act = a * sig
    if not s["backward"]:
        h = w * act * b
        return _rows8(h) if s["fp8"] else h.to(dtype)
    d = s["grad"].float()
    grads = torch.cat([w * d * b * (sig * (1.0 + a * (1.0 - sig))), w * d * act], 1).to(dtype)
    return (grads,) if s["weights"] is None else (grads, (d * act * b).sum(1))


def _blocks(s):
    """Of every row of the sorted list: its route (the number of routes for none) and its row of x."""
    B, n = s["block_m"], s["T"] * s["topk"]
    blocks = s["eid"].numel()
    at = torch.arange(blocks * B, device=DEV)
    sid = torch.where(at < s["npp"], s["sid"][: blocks * B].long(), n)
    row = sid if s["per_route"] else sid // s["topk"]
    return blocks, sid, row.clamp(max=s["x"].shape[0] - 1)


def _experts_plain(s):
    N, K, B, n = s["N"], s["K"], s["block_m"], s["T"] * s["topk"]
    blocks, sid, row = _blocks(s)
    owner = s["eid"].long()
    x = s["x"].float() if s["xs"] is None else s["x"].float() * s["xs"][:, None]
    w = s["w"].float() if s["ws"] is None else s["w"].float() * s["ws"][:, :, None]
    out = getattr(torch, s["out"])
    if not s["backward"]:
        y = torch.bmm(x[row].reshape(blocks, B, K), w[owner].transpose(1, 2)).reshape(blocks * B, N)
        if s["weighted"]:
            y = y * s["sw"][: blocks * B, None]
        return torch.zeros(n + 1, N, device=DEV).index_copy_(0, sid, y)[:n].to(out)
    g = torch.cat([s["grad"].float(), torch.zeros(1, N, device=DEV)])[sid].reshape(blocks, B, N)
    rows = torch.zeros(n + 1, K, device=DEV).index_copy_(0, sid, torch.bmm(g, w[owner]).reshape(blocks * B, K))[:n]
    each = torch.bmm(g.transpose(1, 2), x[row].reshape(blocks, B, K))  # of the rows without a route: zero
    return {"rows": rows.to(s["x"].dtype), "weights": torch.zeros(s["E"], N, K, device=DEV).index_add_(0, owner, each).to(out)}


# -------------------------------------------------------------------- the package's calls
def _own_norm(s, mrs):
    kept, dtype = s["kept"], getattr(torch, s["dtype"])
    if not s["backward"]:
        if not kept:
            kept["out"] = mrs.NormBuffers.allocate(s["T"], s["cols"], dtype, sum=True, fp8=s["fp8"], device=DEV)
        out = mrs.rms_norm(s["x"], s["gain"], EPS, residual=s["residual"], parts=s["parts"], out=kept["out"])
        if not s["fp8"]:
            return {"y": out.y, "sum": out.sum}
        return {"y": out.y, "sum": out.sum, "codes": out.rows8.codes, "scales": out.rows8.scales}
    if not kept:
        kept["out"] = mrs.NormGrads.allocate(s["T"], s["cols"], dtype, device=DEV)
    out = mrs.rms_norm_backward(s["s"], s["gain"], s["rstd"], grad=s["grad"], grad_rows=s["grad_rows"], parts=s["parts"], grad_sum=s["grad_sum"],
                                out=kept["out"])
    return {"grad_x": out.x, "grad_gain": out.weight}


def _own_gated(s, mrs):
    kept = s["kept"]
    if not s["backward"]:
        if not kept:
            kept["out"] = mrs.Fp8Rows.allocate(s["rows"], s["cols"], device=DEV) if s["fp8"] else torch.empty_like(s["x"][:, : s["cols"]])
        h = mrs.swiglu(s["x"], s["weights"], out=kept["out"])
        return (h.codes, h.scales) if s["fp8"] else h
    if not kept:
        kept["out"] = (torch.empty_like(s["x"]), None if s["weights"] is None else torch.empty_like(s["weights"]))
    grads, weights = mrs.swiglu_backward(s["grad"], s["x"], s["weights"], out=kept["out"])
    return (grads,) if weights is None else (grads, weights)


def _own(s):
    import moe_expert_routing_sort_gb300 as mrs

    if s["op"] == "norm":
        return _own_norm(s, mrs)
    if s["op"] == "gated":
        return _own_gated(s, mrs)
    kept, n, out = s["kept"], s["T"] * s["topk"], getattr(torch, s["out"])
    if not kept:  # the outputs' buffers, cleared once: rows of dropped routes are not written
        kept["ws"] = mrs.ProductWorkspace.allocate(s["T"], s["E"], s["topk"], s["block_m"], device=DEV)
        kept["x"] = s["x"] if s["xs"] is None else mrs.Fp8Rows(s["x"], s["xs"])
        kept["w"] = s["w"] if s["ws"] is None else mrs.Fp8Rows(s["w"], s["ws"])
        kept["rows"] = torch.zeros(n, s["K"] if s["backward"] else s["N"], dtype=s["x"].dtype if s["backward"] else out, device=DEV)
        if s["backward"]:
            kept["weights"] = torch.empty(s["E"], s["N"], s["K"], dtype=out, device=DEV)
    routes = (s["T"], s["topk"], s["block_m"], s["sid"], s["eid"], s["npp"])
    if not s["backward"]:
        return mrs.experts_product(kept["x"], kept["w"], *routes, sorted_weights=s["sw"] if s["weighted"] else None, out=kept["rows"],
                                   workspace=kept["ws"])
    return {"rows": mrs.experts_grad_rows(s["grad"], s["w"], *routes, out=kept["rows"], workspace=kept["ws"]),
            "weights": mrs.experts_grad_weights(s["grad"], s["x"], s["E"], *routes, out=kept["weights"], workspace=kept["ws"])}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "norm":
        return _norm_plain(state)
    if state["op"] == "gated":
        return _gated_plain(state)
    return _experts_plain(state)


# ------------------------------------------------------------------------- what it takes
def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["cols"]
        if c["backward"]:
            return {"bytes": 2 * n * (c["parts"] + 4) + 4 * c["T"] + 6 * c["cols"], "flops": n * (c["parts"] + 10)}
        return {"bytes": n * (2 * (c["parts"] + 3) + c["fp8"]) + 4 * c["T"] * c["fp8"] + 2 * c["cols"], "flops": n * (c["parts"] + 5)}
    if c["op"] == "gated":
        n, weights = c["rows"] * c["cols"], 4 * c["rows"] * c["weighted"]
        if c["backward"]:
            return {"bytes": 10 * n + 2 * weights, "flops": 16 * n}
        return {"bytes": n * (5 if c["fp8"] else 6) + 4 * c["rows"] * c["fp8"] + weights, "flops": 7 * n}
    T, E, topk, K, N = c["T"], c["E"], c["topk"], c["K"], c["N"]
    routes = T * topk * (0.9 if c["drop"] else 1.0)
    hit = min(float(T * topk), E * (1.0 - (1.0 - topk / E) ** T))  # experts with any row
    size, out = 1 if c["dtype"] == "float8_e4m3fn" else 2, 4 if c["out"] == "float32" else 2
    rows = T * topk if c["per_route"] else T
    if c["backward"]:
        # weights, both sides' rows (the gradients for both products), the rows' and the weights' gradients
        return {"bytes": 2 * hit * N * K + 2 * routes * N + 2 * rows * K + 2 * routes * K + out * E * N * K, "flops": 4.0 * routes * N * K}
    return {"bytes": size * (hit * N * K + rows * K) + routes * N * out + (4 * (hit * N + rows) if size == 1 else 0), "flops": 2.0 * routes * N * K}


# ------------------------------------------------------- from the definitions, in 64 bits
def _exact_rows8(y):
    """Codes' values and scales of rows in 64 bits: the nearest of the e4m3 grid, ties to even."""
    scale = (y.abs().amax(1, keepdim=True) / TOP).clamp(min=TINY)
    v = (y / scale).abs()
    e = torch.frexp(v.clamp(min=2.0 ** -7)).exponent - 1  # binade, the subnormals' one at least
    step = torch.ldexp(torch.ones_like(v), (e.clamp(min=-6) - 3))
    return torch.sign(y) * (torch.round(v / step) * step).clamp(max=TOP), scale[:, 0]


def _exact_norm(s):
    T, cols, parts = s["T"], s["cols"], s["parts"]
    gain = s["gain"].double()
    if not s["backward"]:
        total = s["residual"].double()
        for j in range(parts):
            total = total + s["x"][j::parts].double()
        t = total.to(s["residual"].dtype).double()
        y = t * gain / torch.sqrt(t.pow(2).sum(1, keepdim=True) / cols + EPS)
        codes, scales = _exact_rows8(y)
        return {"y": y, "sum": total, "codes": codes, "scales": scales} if s["fp8"] else {"y": y, "sum": total}
    # by differentiating the definition, with the reciprocal root that the caller kept
    d = s["grad"].double()
    for j in range(parts):
        d = d + s["grad_rows"][j::parts].double()
    r = s["rstd"].double()[:, None]
    xh = s["s"].double() * r
    dx = d * gain * r - xh * r * ((d * gain * xh).sum(1, keepdim=True) / cols) + s["grad_sum"].double()
    return {"grad_x": dx, "grad_gain": (d * xh).sum(0)}


def _exact_gated(s):
    cols = s["cols"]
    x = s["x"].double().requires_grad_()
    w = torch.ones(s["rows"], dtype=torch.float64, device=DEV) if s["weights"] is None else s["weights"].double()
    w.requires_grad_()
    h = w[:, None] * x[:, :cols] * torch.sigmoid(x[:, :cols]) * x[:, cols:]
    if not s["backward"]:
        return _exact_rows8(h.detach()) if s["fp8"] else h.detach()
    grads = torch.autograd.grad(h, (x, w), s["grad"].double())
    return grads[:1] if s["weights"] is None else grads


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        return _exact_norm(s)
    if s["op"] == "gated":
        return _exact_gated(s)
    T, E, topk, N, K, B = s["T"], s["E"], s["topk"], s["N"], s["K"], s["block_m"]
    if (4.0 if s["backward"] else 2.0) * T * topk * N * K > 8e12:
        return None
    used = int(s["npp"])
    sid = s["sid"][:used].long()
    owner = s["eid"][: used // B].long().repeat_interleave(B)
    rows = torch.zeros(T * topk, K if s["backward"] else N, dtype=torch.float64, device=DEV)
    weights = torch.zeros(E, N, K, dtype=torch.float64, device=DEV) if s["backward"] else None
    for e in owner.unique().tolist():
        at = ((owner == e) & (sid < T * topk)).nonzero()[:, 0]
        r = sid[at]
        i = r if s["per_route"] else torch.div(r, topk, rounding_mode="floor")
        x, w = s["x"][i].double(), s["w"][e].double()
        if s["xs"] is not None:
            x, w = x * s["xs"][i].double()[:, None], w * s["ws"][e].double()[:, None]
        if s["backward"]:
            g = s["grad"][r].double()
            rows[r] = g @ w
            weights[e] = g.T @ x
        else:
            y = x @ w.T
            rows[r] = y * s["sw"][at].double()[:, None] if s["weighted"] else y
    return {"rows": rows, "weights": weights} if s["backward"] else rows
