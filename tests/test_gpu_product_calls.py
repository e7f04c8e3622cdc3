"""Calls of the experts' products and of the operators around them, as programs make them: whole
layers, graphs, streams, long lists, lists that are not in order, waits that give up, NaN in other
tokens' rows, offsets past 32 bits.  Tolerances as in test_gpu_products.py and test_gpu_rows.py."""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs
from test_gpu_products import BF, DEV, F32, FH, Routes, _gen, _near, _per_route, _ref, _rows
from test_gpu_rows import HALF, U, _close, _close8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


# ------------------------------------------------------------------ more shapes and paths
# T, E, topk, cols, outs, block_m: two tiles of outputs on the same rows; odd numbers of them; lists
# that a kernel of its own cuts, with narrow and wide tiles; blocks of one row; many experts
PATHS = [
    (600, 2, 2, 1160, 648, 64),
    (500, 3, 1, 2064, 1000, 16),
    (3000, 2000, 2, 72, 136, 16),
    (4000, 1100, 16, 64, 72, 16),
    (5000, 8, 2, 64, 72, 1),
    (300, 4096, 4, 32, 264, 32),
    (129, 1, 1, 80, 40, 16),
    (128, 1, 1, 80, 40, 1024),
    (9, 2, 2, 4160, 40, 64),
    (4096, 8, 2, 2064, 5128, 64),
    (4096, 8, 2, 5136, 1032, 64),
    (4000, 1100, 16, 64, 3592, 16),  # several output tiles a unit, wide and narrow row tiles
    (3000, 2000, 2, 72, 1544, 16),
]


@pytest.mark.parametrize("T,E,topk,cols,outs,B", PATHS)
def test_paths(T, E, topk, cols, outs, B):
    g = _gen("x", T, E, cols, outs)
    r = Routes(g, T, E, topk, B, "skewed")
    w = _rows(g, E * outs, cols, BF).view(E, outs, cols)
    ws = mrs.ProductWorkspace(T, E, topk, B, device=DEV)
    x, grad = _rows(g, T, cols, BF), _rows(g, T * topk, outs, BF)
    y = mrs.experts_product(x, w, *r.lists, dtype=F32, workspace=ws)
    _near(y, *_ref(x, w, r), cols, 1)
    if cols % 16 == 0:
        x8, w8 = mrs.fp8_quantize(x), mrs.fp8_quantize(w)
        y8 = mrs.experts_product(x8, w8, *r.lists, sorted_weights=r.sw, workspace=ws)
        want, size = _ref(x8.codes.double() * x8.scales.double()[:, None],
                          w8.codes.double() * w8.scales.double()[..., None], r)
        by = r.weights.reshape(-1, 1).double()
        _near(y8, want * by, size * by, cols, 4)
    dx = mrs.experts_grad_rows(grad, w, *r.lists, dtype=F32, workspace=ws)
    _near(dx, *_ref(grad, w.transpose(1, 2), r), outs)
    dw = mrs.experts_grad_weights(grad, x, E, *r.lists, workspace=ws)
    gd, xd, owner = grad.double(), _per_route(x, r).double(), r.owners()
    for e in range(E):
        at = (owner == e).nonzero()[:, 0]
        _near(dw[e], gd[at].T @ xd[at], gd[at].T.abs() @ xd[at].abs(), max(at.numel(), 1))
    assert ws.status_word() == 0


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "rows"])
def test_wide_outputs_over_many_rounds(kind, dtype):
    """Outputs (or the gradient's columns) that leave a pair of CTAs more than 40 tiles, which are
    then of 512 outputs.  Checked at both ends and in 400 places."""
    T, E, topk, B, wide, deep = 3000, 2, 2, 64, 41416, 2080 if kind == "fp8" else 1040
    g = _gen("rounds", kind)
    r = Routes(g, T, E, topk, B)
    pick = torch.cat([torch.arange(300, device=DEV), torch.arange(wide - 300, wide, device=DEV),
                      torch.randperm(wide, generator=g, device=DEV)[:400]])
    ws = mrs.ProductWorkspace(T, E, topk, B, device=DEV)
    terms = 4 if kind == "fp8" else 1
    if kind == "rows":
        w = _rows(g, E * deep, wide, BF).view(E, deep, wide)
        x = _rows(g, T * topk, deep, BF)
        y = mrs.experts_grad_rows(x, w, *r.lists, dtype=dtype, workspace=ws)
        want, size = _ref(x, w.transpose(1, 2)[:, pick], r)
    else:
        x, w = _rows(g, T, deep, BF), _rows(g, E * wide, deep, BF).view(E, wide, deep)
        if kind == "fp8":
            x, w = mrs.fp8_quantize(x), mrs.fp8_quantize(w)
        y = mrs.experts_product(x, w, *r.lists, dtype=dtype, workspace=ws)
        if kind == "fp8":
            x = x.codes.double() * x.scales.double()[:, None]
            w = w.codes.double()[:, pick] * w.scales.double()[:, pick, None]
        else:
            w = w[:, pick]
        want, size = _ref(x, w, r)
    _near(y[:, pick], want, size, deep, terms)
    assert ws.status_word() == 0


def test_results_are_the_same_bits_every_call():
    g = _gen("same")
    r = Routes(g, 700, 9, 4, 32, "skewed")
    w, x, grad = _rows(g, 9 * 264, 520, BF).view(9, 264, 520), _rows(g, 700, 520, BF), None
    grad = _rows(g, 2800, 264, BF)
    first = None
    for _ in range(4):
        got = (mrs.experts_product(x, w, *r.lists, dtype=F32),
               mrs.experts_grad_rows(grad, w, *r.lists, dtype=F32),
               mrs.experts_grad_weights(grad, x, 9, *r.lists))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


# ----------------------------------------------------------------------------- whole layers
def test_a_layer_served_in_8_bits():
    """norm -> router -> first product -> gated activation -> second product -> next norm, each step
    checked against its definition on the rows that it got."""
    T, E, topk, cols, inter, B, scale = 37, 16, 4, 256, 96, 16, 2.5
    g = _gen("serve")
    hidden, delta = _rows(g, T, cols, BF), _rows(g, T, cols, BF)
    gain, gain2 = _rows(g, 2, cols, BF) + 1
    gate = _rows(g, E, cols, BF, 0.1)
    up = mrs.fp8_quantize(_rows(g, E * 2 * inter, cols, F32, 0.1).view(E, 2 * inter, cols))
    down = mrs.fp8_quantize(_rows(g, E * cols, inter, F32, 0.1).view(E, cols, inter))
    n = mrs.rms_norm(delta, gain, residual=hidden, sum=True, fp8=True)
    logits = (n.y.float() @ gate.float().T).bfloat16()
    r = mrs.route_sort(logits, torch.zeros(E, device=DEV), 1, 1, topk, scale, B)
    lists = (T, topk, B, r.sorted_token_ids, r.expert_ids, r.num_tokens_post_pad)
    ws = mrs.ProductWorkspace.allocate(T, E, topk, B, device=DEV)
    a = mrs.experts_product(n.rows8, up, *lists, workspace=ws)
    h = mrs.swiglu(a, fp8=True)
    y = mrs.experts_product(h, down, *lists, sorted_weights=r.sorted_weights, workspace=ws)
    out = mrs.rms_norm(y, gain2, residual=n.sum, parts=topk, sum=True)
    assert ws.status_word() == 0

    class R:
        pass

    q = R()
    q.T, q.topk, q.owners = T, topk, lambda: r.topk_ids.reshape(-1).long()

    def values(rows8):
        return rows8.codes.double() * rows8.scales.double()[..., None]

    s = n.sum.double()
    assert torch.equal(n.sum, (hidden.float() + delta.float()).bfloat16())
    _close8(n.rows8, s * gain.double() / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-6), 48 * U)
    _near(a, *_ref(values(n.rows8), values(up), q), cols, 4)
    ad = a.double()
    _close8(h, ad[:, :inter] * torch.sigmoid(ad[:, :inter]) * ad[:, inter:], 240 * U)
    by = r.topk_weights.reshape(-1, 1).double()
    want, size = _ref(values(h), values(down), q)
    _near(y, want * by, size * by, inter, 4)
    total = n.sum.double() + y.double().view(T, topk, cols).sum(1)
    _close(out.sum, total, (topk + 1) * U * (n.sum.double().abs() +
                                             y.double().abs().view(T, topk, cols).sum(1)), BF)


def test_a_layer_trained():
    """The forward pass of a layer and the gradient of all it is made of, each step checked against
    its definition, and the routing weights' gradient handed to the router's."""
    T, E, topk, cols, inter, B, scale = 50, 12, 3, 128, 72, 16, 1.5
    g = _gen("train")
    hidden = _rows(g, T, cols, BF)
    gain, gate = _rows(g, 1, cols, BF)[0] + 1, _rows(g, E, cols, BF, 0.2)
    up = _rows(g, E * 2 * inter, cols, BF, 0.1).view(E, 2 * inter, cols)
    down = _rows(g, E * cols, inter, BF, 0.1).view(E, cols, inter)
    n = mrs.rms_norm(hidden, gain, sum=True, rstd=True)
    logits = (n.y.float() @ gate.float().T).bfloat16()
    r = mrs.route_sort_softmax(logits, topk, scale, B)
    lists = (T, topk, B, r.sorted_token_ids, r.expert_ids, r.num_tokens_post_pad)
    weights = r.topk_weights.reshape(-1)
    a = mrs.experts_product(n.y, up, *lists)
    h = mrs.swiglu(a, weights)
    y = mrs.experts_product(h, down, *lists)
    # the layer's output is the sum of a token's rows: its gradient reaches every one of them
    dout = _rows(g, T, cols, BF)
    dh = mrs.experts_grad_rows(dout, down, *lists)
    ddown = mrs.experts_grad_weights(dout, h, E, *lists)
    da, dweights = mrs.swiglu_backward(dh, a, weights)
    dy = mrs.experts_grad_rows(da, up, *lists)
    dup = mrs.experts_grad_weights(da, n.y, E, *lists)
    dlogits = mrs.route_backward(logits, r.topk_ids, dweights.view(T, topk), scale, softmax=True)
    dy_router = (dlogits.float() @ gate.float()).bfloat16()
    grads = mrs.rms_norm_backward(n.sum, gain, n.rstd, grad=dy_router, grad_rows=dy, parts=topk,
                                  grad_sum=dout)

    class R:
        pass

    q = R()
    q.T, q.topk, q.owners = T, topk, lambda: r.topk_ids.reshape(-1).long()
    owner = q.owners()
    _near(a, *_ref(n.y, up, q), cols)
    _near(y, *_ref(h, down, q), inter)
    _near(dh, *_ref(dout, down.transpose(1, 2), q), cols)
    _near(dy, *_ref(da, up.transpose(1, 2), q), 2 * inter)
    for got, u, v in ((ddown, _per_route(dout, q), h), (dup, da, _per_route(n.y, q))):
        u, v = u.double(), v.double()
        for e in range(E):
            at = (owner == e).nonzero()[:, 0]
            _near(got[e], u[at].T @ v[at], u[at].T.abs() @ v[at].abs(), max(at.numel(), 1))
    # the chain of the weights: by differentiating in float64 what the activation computes
    ad = a.double().requires_grad_()
    wd = weights.double().requires_grad_()
    hd = wd[:, None] * torch.nn.functional.silu(ad[:, :inter]) * ad[:, inter:]
    ga, gw = torch.autograd.grad(hd, (ad, wd), dh.double())
    assert ((da.double() - ga).abs() <= HALF[BF] * ga.abs() + 2.0**-18 * ga.abs().amax()).all()
    assert ((dweights.double() - gw).abs() <= 2.0**-17 * (dh.double() * hd / wd[:, None]).abs().sum(1)).all()
    xd = logits.double().requires_grad_()
    p = torch.softmax(xd.gather(1, r.topk_ids.long()), 1) * scale
    want = torch.autograd.grad(p, xd, dweights.double().view(T, topk))[0]
    assert ((dlogits.double() - want).abs() <= HALF[BF] * want.abs() + 1e-5 * want.abs().amax()).all()
    sd = n.sum.double().requires_grad_()
    yd = sd / torch.sqrt(sd.square().mean(1, keepdim=True) + 1e-6) * gain.double()
    up_to = dy_router.double() + dy.double().view(T, topk, cols).sum(1)
    gs = torch.autograd.grad(yd, sd, up_to)[0] + dout.double()
    # sums of 128 terms in fp32, a handful of levels: 2^-17 of the largest term
    most = (up_to.abs() * gain.double().abs()).amax() * n.rstd.double().amax() * 8
    assert ((grads.x.double() - gs).abs() <= HALF[BF] * gs.abs() + 2.0**-17 * most).all()


# ------------------------------------------------------------------------ graphs and streams
def test_captured_and_replayed_on_new_rows():
    g = _gen("graph")
    for T, E, topk, B in ((3, 6, 2, 16), (40, 6, 2, 16), (900, 6, 2, 64)):
        r = Routes(g, T, E, topk, B)
        w = _rows(g, E * 264, 136, BF).view(E, 264, 136)
        x, grad = _rows(g, T, 136, BF), _rows(g, T * topk, 264, BF)
        ws = mrs.ProductWorkspace(T, E, topk, B, device=DEV)
        y = torch.zeros(T * topk, 264, dtype=BF, device=DEV)
        dx, dw = torch.zeros(T * topk, 136, dtype=BF, device=DEV), torch.zeros_like(w)

        def calls():
            mrs.experts_product(x, w, *r.lists, sorted_weights=r.sw, out=y, workspace=ws)
            mrs.experts_grad_rows(grad, w, *r.lists, out=dx, workspace=ws)
            mrs.experts_grad_weights(grad, x, E, *r.lists, out=dw, workspace=ws)

        calls()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        for _ in range(3):
            x.copy_(_rows(g, T, 136, BF))
            grad.copy_(_rows(g, T * topk, 264, BF))
            calls()
            want = [t.clone() for t in (y, dx, dw)]
            for t in (y, dx, dw):
                t.fill_(7.0)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(want, (y, dx, dw)))
        assert ws.status_word() == 0


def test_two_graphs_at_once_with_a_workspace_each():
    g = _gen("two")
    jobs = []
    for T, E in ((700, 1500), (800, 1400)):  # (lists that a kernel cuts into the workspace)
        r = Routes(g, T, E, 4, 16)
        w, x = _rows(g, E * 136, 72, BF).view(E, 136, 72), _rows(g, T, 72, BF)
        ws = mrs.ProductWorkspace(T, E, 4, 16, device=DEV)
        y = torch.zeros(T * 4, 136, dtype=BF, device=DEV)
        mrs.experts_product(x, w, *r.lists, out=y, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                mrs.experts_product(x, w, *r.lists, out=y, workspace=ws)
        jobs.append((graph, y, y.clone(), torch.cuda.Stream(), ws, (r, w, x)))
    for _ in range(5):
        torch.cuda.synchronize()
        for graph, y, _, stream, *_ in jobs:
            with torch.cuda.stream(stream):
                y.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for _, y, want, _, ws, _ in jobs:
            assert torch.equal(y, want) and ws.status_word() == 0


def test_on_another_stream_without_buffers():
    g = _gen("stream")
    r = Routes(g, 400, 8, 2, 32)
    w, x = _rows(g, 8 * 136, 200, FH).view(8, 136, 200), _rows(g, 400, 200, FH)
    grad = _rows(g, 800, 136, FH)
    want = (mrs.experts_product(x, w, *r.lists), mrs.experts_grad_rows(grad, w, *r.lists),
            mrs.experts_grad_weights(grad, x, 8, *r.lists))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        got = (mrs.experts_product(x, w, *r.lists, stream=handle),
               mrs.experts_grad_rows(grad, w, *r.lists, stream=handle),
               mrs.experts_grad_weights(grad, x, 8, *r.lists, stream=handle))
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


# --------------------------------------------------------------- lists that are not in order
class Guarded:
    """A buffer between marks."""

    def __init__(self, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        self.all = torch.full((n + 8192,), 7.0, dtype=dtype, device=DEV)
        self.t = self.all[4096:4096 + n].view(shape)

    def untouched_around(self):
        n = self.t.numel()
        return bool((self.all[:4096] == 7).all()) and bool((self.all[4096 + n:] == 7).all())


@pytest.mark.parametrize("T,E,topk,B", [(5, 4, 2, 16), (200, 4, 2, 16), (700, 4, 3, 64),
                                        (700, 1500, 4, 16)])
@pytest.mark.parametrize("how", ["past", "negative", "descending"])
def test_owners_out_of_order_are_reported(T, E, topk, B, how):
    g = _gen("bad", T, E)
    r = Routes(g, T, E, topk, B)
    used = int(r.npp) // B
    eid = r.eid.clone()
    at = used // 2
    if how == "descending":
        eid[:used] = eid[:used].flip(0)
    else:
        eid[at] = E + 5 if how == "past" else -1
    w, x = _rows(g, E * 72, 40, BF).view(E, 72, 40), _rows(g, T, 40, BF)
    grad = _rows(g, T * topk, 72, BF)
    lists = (T, topk, B, r.sid, eid, r.npp)
    ws = mrs.ProductWorkspace(T, E, topk, B, device=DEV)
    y, dx, dw = Guarded((T * topk, 72), BF), Guarded((T * topk, 40), BF), Guarded((E, 72, 40), F32)
    for call in (lambda: mrs.experts_product(x, w, *lists, out=y.t, workspace=ws),
                 lambda: mrs.experts_grad_rows(grad, w, *lists, out=dx.t, workspace=ws),
                 lambda: mrs.experts_grad_weights(grad, x, E, *lists, out=dw.t, workspace=ws)):
        call()
        assert ws.status_word() == mrs.DEVICE_BAD_EXPERT_ID
        ws.clear()
    for buf in (y, dx, dw):
        assert buf.untouched_around()
    # and the next call is a call as any other
    good = mrs.experts_product(x, w, *r.lists, dtype=F32, workspace=ws)
    _near(good, *_ref(x, w, r), 40, 1)
    assert ws.status_word() == 0


def test_entries_of_the_list_that_are_no_route():
    # behind the routes of a block anything that is no route is padding
    g = _gen("pad")
    r = Routes(g, 300, 4, 2, 32)
    w, x, grad = _rows(g, 4 * 72, 40, BF).view(4, 72, 40), _rows(g, 300, 40, BF), _rows(g, 600, 72, BF)
    want = (mrs.experts_product(x, w, *r.lists), mrs.experts_grad_rows(grad, w, *r.lists),
            mrs.experts_grad_weights(grad, x, 4, *r.lists))
    pads = (r.sid == 600).nonzero()[:, 0]
    sid = r.sid.clone()
    sid[pads] = torch.where(pads % 2 == 0, -5, 2**31 - 1).int()
    lists = (300, 2, 32, sid, r.eid, r.npp)
    got = (mrs.experts_product(x, w, *lists), mrs.experts_grad_rows(grad, w, *lists),
           mrs.experts_grad_weights(grad, x, 4, *lists))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # a length of zero, and one past the list
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = torch.full((600, 72), 7.0, dtype=BF, device=DEV)
    mrs.experts_product(x, w, 300, 2, 32, r.sid, r.eid, none, out=y)
    assert (y == 7).all()
    assert not mrs.experts_grad_weights(grad, x, 4, 300, 2, 32, r.sid, r.eid, none).any()


def test_waits_that_give_up_are_reported():
    g = _gen("wait")
    for T, topk in ((4, 2), (300, 2), (3000, 2)):
        r = Routes(g, T, 6, topk, 16)
        w, x = _rows(g, 6 * 72, 136, BF).view(6, 72, 136), _rows(g, T, 136, BF)
        grad = _rows(g, T * topk, 72, BF)
        ws = mrs.ProductWorkspace(T, 6, topk, 16, device=DEV)
        y, dx, dw = Guarded((T * topk, 72), BF), Guarded((T * topk, 136), BF), Guarded((6, 72, 136), BF)
        mrs.moe_route_sort_debug_set(mrs.DEBUG_WAIT_LIMIT_NS, 0)
        try:
            for call in (lambda: mrs.experts_product(x, w, *r.lists, out=y.t, workspace=ws),
                         lambda: mrs.experts_grad_rows(grad, w, *r.lists, out=dx.t, workspace=ws),
                         lambda: mrs.experts_grad_weights(grad, x, 6, *r.lists, out=dw.t,
                                                          workspace=ws)):
                call()
                assert ws.status_word() == mrs.DEVICE_WAIT_TIMEOUT
                ws.clear()
        finally:
            mrs.moe_route_sort_debug_set(mrs.DEBUG_WAIT_LIMIT_NS, -1)
        assert all(b.untouched_around() for b in (y, dx, dw))
        _near(mrs.experts_product(x, w, *r.lists, dtype=F32, workspace=ws), *_ref(x, w, r), 136, 1)
        assert ws.status_word() == 0


# ----------------------------------------------------------------------- NaN of other tokens
def test_nan_stays_with_its_token():
    g = _gen("nan")
    for T, topk in ((6, 2), (90, 2), (900, 2)):
        E = 3
        r = Routes(g, T, E, topk, 16)
        w, x = _rows(g, E * 136, 72, BF).view(E, 136, 72), _rows(g, T, 72, BF)
        grad = _rows(g, T * topk, 136, BF)
        # tensor memory and shared memory full of NaN, as another call may leave them
        full = torch.full_like(x, float("nan"))
        mrs.experts_product(full, w, *r.lists)
        mrs.experts_grad_weights(torch.full_like(grad, float("nan")), full, E, *r.lists)
        x[0] = float("nan")
        x[T // 2] = float("inf")
        bad = torch.zeros(T, dtype=torch.bool, device=DEV)
        bad[0] = bad[T // 2] = True
        y = mrs.experts_product(x, w, *r.lists, dtype=F32)
        ok = ~bad.repeat_interleave(topk)
        want, size = _ref(torch.where(bad[:, None], 0.0, x.float()), w, r)
        _near(y[ok], want[ok], size[ok], 72, 1)
        assert not torch.isfinite(y[~ok]).any()
        dw = mrs.experts_grad_weights(grad, x, E, *r.lists)
        hit = r.ids[bad].unique().long()
        for e in range(E):
            at = (r.owners() == e).nonzero()[:, 0]
            if (hit == e).any():
                assert not torch.isfinite(dw[e]).all()
            else:
                gd, xd = grad.double()[at], _per_route(x, r).double()[at]
                _near(dw[e], gd.T @ xd, gd.T.abs() @ xd.abs(), max(at.numel(), 1))
        dx = mrs.experts_grad_rows(grad, w, *r.lists, dtype=F32)
        _near(dx, *_ref(grad, w.transpose(1, 2), r), 136)


# ------------------------------------------------------------------------------ large tensors
def test_rows_and_outputs_past_32_bit_offsets():
    g = _gen("far")
    T, cols = 33000, 65536
    r = Routes(g, T, 1, 1, 128)
    last = torch.arange(T - 3, T, device=DEV)
    x = torch.zeros(T, cols, dtype=BF, device=DEV)  # 4.3 GB, 2.2e9 elements
    x[last] = _rows(g, 3, cols, BF)
    w = _rows(g, 72, cols, BF).view(1, 72, cols)
    y = mrs.experts_product(x, w, *r.lists, dtype=F32)
    want, size = x[last].double() @ w[0].double().T, x[last].double().abs() @ w[0].double().abs().T
    _near(y[last], want, size, cols, 1)
    assert not y[:-3].any()
    grad = _rows(g, T, 72, BF)
    dw = mrs.experts_grad_weights(grad, x, 1, *r.lists)
    gd, xd = grad[last].double(), x[last].double()
    _near(dw[0], gd.T @ xd, gd.T.abs() @ xd.abs(), T)
    dx = mrs.experts_grad_rows(grad, w, *r.lists)
    _near(dx[last], grad[last].double() @ w[0].double(),
          grad[last].double().abs() @ w[0].double().abs(), 72)


def test_gradient_of_weights_over_thousands_of_rows():
    """Experts of up to 5000 rows, at and beside the numbers from which tiles are summed in two parts,
    each with several tiles for a pair of CTAs."""
    g = _gen("long")
    counts, cols, outs = (1000, 5000, 4097, 0, 4096, 1024, 1025), 2056, 1288
    T = sum(counts)
    r = Routes(g, T, len(counts), 1, 16)
    owner = torch.cat([torch.full((n,), e, device=DEV) for e, n in enumerate(counts)])
    r.ids = owner[torch.randperm(T, generator=g, device=DEV)].int().view(T, 1)
    ws = torch.zeros(mrs.moe_route_sort_workspace_bytes(T, r.E, 1, 16), dtype=torch.uint8,
                     device=DEV)
    mrs.moe_sort(r.ids, r.weights, r.E, 16, r.sid, r.sw, r.eid, r.npp, ws)
    x, grad = _rows(g, T, cols, FH), _rows(g, T, outs, FH)
    owner = r.owners()
    for kind in (F32, FH):
        dw = mrs.experts_grad_weights(grad, x, len(counts), *r.lists, dtype=kind)
        for e, n in enumerate(counts):
            at = (owner == e).nonzero()[:, 0]
            assert at.numel() == n
            gd, xd = grad[at].double(), x[at].double()
            _near(dw[e], gd.T @ xd, gd.T.abs() @ xd.abs(), max(n, 1))


def test_long_sums_stay_near_fp32():
    """An addition to an accumulator takes 16 products and cuts what is below its last bit, half of
    that bit on average: at most 2^-24 of the sum so far.  The sums on the way to a sum of n random
    terms have n / 2 in common with it on average, so that it is low by n / 16 / 2 * 2^-24 at most.
    Two accumulators have half of the rows each."""
    n = 8192
    g = _gen("low")
    r = Routes(g, n, 1, 1, 16)
    x, grad = _rows(g, n, 256, FH), _rows(g, n, 256, FH)
    want = grad.double().T @ x.double()
    dw = mrs.experts_grad_weights(grad, x, 1, *r.lists, dtype=F32)
    assert ((dw[0].double() - want).norm() / want.norm()).item() <= n / 2 / 16 / 2 * 2**-24


def test_weights_past_32_bit_offsets():
    g = _gen("heavy")
    E, outs, cols = 68, 512, 65536  # 2.3e9 elements
    w = torch.zeros(E, outs, cols, dtype=BF, device=DEV)
    w[-1] = _rows(g, outs, cols, BF)
    for T in (20, 300):
        ids = torch.full((T, 1), E - 1, dtype=torch.int32, device=DEV)
        r = Routes(g, T, E, 1, 16)
        ws = torch.zeros(mrs.moe_route_sort_workspace_bytes(T, E, 1, 16), dtype=torch.uint8, device=DEV)
        mrs.moe_sort(ids, r.weights, E, 16, r.sid, r.sw, r.eid, r.npp, ws)
        r.ids = ids
        x, grad = _rows(g, T, cols, BF), _rows(g, T, outs, BF)
        xd, wd = x.double(), w[-1].double()
        _near(mrs.experts_product(x, w, *r.lists, dtype=F32), xd @ wd.T, xd.abs() @ wd.abs().T, cols, 1)
        gd = grad.double()
        _near(mrs.experts_grad_rows(grad, w, *r.lists), gd @ wd, gd.abs() @ wd.abs(), outs)
    dw = mrs.experts_grad_weights(grad, x, E, *r.lists, dtype=BF)
    assert not dw[:-1].any()
    _near(dw[-1], gd.T @ xd, gd.T.abs() @ xd.abs(), T)


# ---------------------------------------------------------------------------------- refusals
def test_refusals_on_the_device():
    x, w = torch.zeros(4, 64, dtype=BF, device=DEV), torch.zeros(2, 16, 64, dtype=BF, device=DEV)
    i = torch.zeros(64, dtype=torch.int32, device=DEV)
    grad = torch.zeros(8, 16, dtype=BF, device=DEV)
    lists = (4, 2, 16, i, i, i)
    cases = [
        (lambda: mrs.experts_product(x.half(), w, *lists), "x must be torch.bfloat16"),
        (lambda: mrs.experts_product(x[:3], w, *lists), "x must be .T = 4"),
        (lambda: mrs.experts_product(x[:, :32].contiguous(), w, *lists), "x must be"),
        (lambda: mrs.experts_product(x, w.float(), *lists), "w must be bfloat16 or float16"),
        (lambda: mrs.experts_product(x, w[0], *lists), "E, outs, cols"),
        (lambda: mrs.experts_product(x, w.transpose(1, 2), *lists), "x must be|contiguous"),
        (lambda: mrs.experts_product(x, mrs.fp8_quantize(w), *lists), "x must be Fp8Rows"),
        (lambda: mrs.experts_product(mrs.fp8_quantize(x), w, *lists), "x must be a tensor"),
        (lambda: mrs.experts_product(mrs.fp8_quantize(x[:2]), mrs.fp8_quantize(w), *lists), "x must have"),
        (lambda: mrs.experts_product(x, w, 4, 2, 16, i[:8], i, i), "sorted_token_ids holds"),
        (lambda: mrs.experts_product(x, w, *lists, sorted_weights=torch.zeros(3, device=DEV)),
         "sorted_weights holds"),
        (lambda: mrs.experts_product(x, w, *lists, out=grad[:4]), "out must be .8, 16"),
        (lambda: mrs.experts_product(x, w, *lists, out=grad.double()), "out must be one of"),
        (lambda: mrs.experts_grad_rows(grad[:, :8].contiguous(), w, *lists), "grad must be"),
        (lambda: mrs.experts_grad_weights(grad, x.half(), 2, *lists), "x must be torch.bfloat16"),
        (lambda: mrs.experts_grad_weights(grad, x, 2, *lists, out=torch.zeros(3, 16, 64, device=DEV)),
         "of 2 experts"),
        (lambda: mrs.experts_grad_weights(grad, x, 2, *lists, dtype=FH), "grad_weights must be one of"),
    ]
    for call, match in cases:
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(mrs.RouteSortError):
        mrs.experts_product(x, w, *lists, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(mrs.RouteSortError):
        mrs.experts_product(x[:, :60].contiguous(), w[:, :, :60].contiguous(), *lists)


def test_no_tokens():
    w = torch.zeros(2, 16, 64, dtype=BF, device=DEV)
    i = torch.zeros(0, dtype=torch.int32, device=DEV)
    n = torch.zeros(1, dtype=torch.int32, device=DEV)
    x, grad = torch.zeros(0, 64, dtype=BF, device=DEV), torch.zeros(0, 16, dtype=BF, device=DEV)
    assert mrs.experts_product(x, w, 0, 2, 16, i, i, n).shape == (0, 16)
    assert mrs.experts_grad_rows(grad, w, 0, 2, 16, i, i, n).shape == (0, 64)
    dw = torch.full((2, 16, 64), 7.0, device=DEV)
    mrs.experts_grad_weights(grad, x, 2, 0, 2, 16, i, i, n, out=dw)
    assert not dw.any()
