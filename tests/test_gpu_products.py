"""The experts' products in 16 and 8 bits and their gradients on a GB300, against plain float64
implementations.

A product of two bf16, fp16 or e4m3 values is exact in fp32; a sum of n of them in fp32 is within
n * 2^-24 * sum |terms| of the float64 sum in any order, and a matrix unit that keeps at least 24
bits of every aligned term stays within n * 2^-23 * sum |terms|, the tolerance used.  Each factor
(routing weight, a row's scale, an output's scale) adds 2^-24 of the value, a 16-bit output half a
step: 2^-8 of the value in bf16, 2^-11 in fp16 (or half of its smallest step, 2^-25).
"""
import zlib

import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FH, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0**-8, FH: 2.0**-11, F32: 2.0**-24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


def _gen(*key):
    return torch.Generator(device=DEV).manual_seed(zlib.crc32(repr(key).encode()))


class Routes:
    """A sorted list made by moe_sort of random routes."""

    def __init__(self, g, T, E, topk, B, how="uniform"):
        self.T, self.E, self.topk, self.B = T, E, topk, B
        scores = torch.rand(T, E, generator=g, device=DEV)
        if how == "skewed":
            scores = scores ** (1 + 8 * torch.rand(E, generator=g, device=DEV))
        ids = scores.topk(topk, 1).indices.int()
        if how == "one":
            ids = torch.full_like(ids, E // 2)
        if how == "dropped":
            ids = torch.where(torch.rand(T, topk, generator=g, device=DEV) < 0.3, -1, ids)
        if how == "none":
            ids = torch.full_like(ids, -1)
        self.ids = ids.contiguous()
        self.weights = torch.rand(T, topk, generator=g, device=DEV) + 0.1
        P = mrs.moe_sort_max_padded(T, E, topk, B)
        self.sid = torch.full((P,), -7, dtype=torch.int32, device=DEV)
        self.sw = torch.zeros(P, device=DEV)
        self.eid = torch.full((max(P // B, 1),), -7, dtype=torch.int32, device=DEV)
        self.npp = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = torch.zeros(mrs.moe_route_sort_workspace_bytes(T, E, topk, B), dtype=torch.uint8,
                         device=DEV)
        mrs.moe_sort(self.ids, self.weights, E, B, self.sid, self.sw, self.eid, self.npp, ws)
        self.lists = (T, topk, B, self.sid, self.eid, self.npp)

    def owners(self):
        return self.ids.reshape(-1).long()


def _rows(g, n, cols, dtype, scale=1.0):
    return (torch.randn(n, cols, generator=g, device=DEV) * scale).to(dtype)


def _per_route(x, r):
    return x if x.shape[0] == r.T * r.topk else x.repeat_interleave(r.topk, 0)


def _ref(x, w, r):
    """(sums, sums of magnitudes) of each route's product in float64; zeros where it is dropped."""
    x, owner = _per_route(x, r).double(), r.owners()
    out = torch.zeros(2, x.shape[0], w.shape[1], dtype=torch.float64, device=DEV)
    for e in range(w.shape[0]):
        at = (owner == e).nonzero()[:, 0]
        if at.numel():
            out[0, at] = x[at] @ w[e].double().T
            out[1, at] = x[at].abs() @ w[e].double().abs().T
    return out


def _near(got, want, size, terms, factors=0):
    """got is one rounding away from a sum of `terms` terms that are `size` together."""
    slack = terms * 2.0**-23 * size + factors * 2.0**-24 * want.abs()
    room = slack + HALF[got.dtype] * (want.abs() + slack)
    if got.dtype is FH:
        room = room + 2.0**-25
    bad = ~((got.double() - want).abs() <= room)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4],
                                 want[bad][:4])


def _dropped_untouched(out, r, mark):
    gone = (r.owners() < 0).nonzero()[:, 0]
    assert (out[gone] == mark).all()


# T, E, topk, cols, outs, block_m, how
SHAPES = [
    (1, 4, 2, 64, 128, 16, "uniform"),
    (3, 5, 2, 8, 8, 1, "uniform"),
    (1, 896, 16, 256, 264, 16, "uniform"),
    (7, 3, 3, 72, 40, 8, "uniform"),
    (64, 4, 2, 192, 256, 32, "uniform"),
    (100, 7, 3, 136, 520, 16, "dropped"),
    (300, 2, 2, 264, 392, 128, "uniform"),
    (513, 3, 1, 520, 136, 64, "one"),
    (200, 64, 6, 200, 328, 256, "skewed"),
    (700, 5, 4, 1032, 72, 1024, "skewed"),
    (40, 6, 2, 128, 64, 16, "none"),
]


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("T,E,topk,cols,outs,B,how", SHAPES)
def test_product(T, E, topk, cols, outs, B, how, dtype):
    g = _gen("p", T, E, cols, outs)
    r = Routes(g, T, E, topk, B, how)
    w = _rows(g, E * outs, cols, dtype).view(E, outs, cols)
    ws = mrs.ProductWorkspace(T, E, topk, B, device=DEV)
    for per_route, weighted, kind in ((False, False, dtype), (True, True, F32), (True, False, BF),
                                      (False, True, dtype)):
        x = _rows(g, T * topk if per_route else T, cols, dtype)
        out = torch.full((T * topk, outs), 7.0, dtype=kind, device=DEV)
        mrs.experts_product(x, w, *r.lists, sorted_weights=r.sw if weighted else None, out=out,
                            workspace=ws)
        assert ws.status_word() == 0
        want, size = _ref(x, w, r)
        if weighted:
            by = r.weights.reshape(-1, 1).double()
            want, size = want * by, size * by
        routed = r.owners() >= 0
        _near(out[routed], want[routed], size[routed], cols, 1)
        _dropped_untouched(out, r, 7.0)
        fresh = mrs.experts_product(x, w, *r.lists, sorted_weights=r.sw if weighted else None,
                                    dtype=kind)
        assert torch.equal(fresh[routed], out[routed]) and not fresh[~routed].any()


@pytest.mark.parametrize("T,E,topk,cols,outs,B,how", [
    (s[0], s[1], s[2], (s[3] + 15) // 16 * 16, *s[4:]) for s in SHAPES])
def test_product_in_8_bits(T, E, topk, cols, outs, B, how):
    g = _gen("8", T, E, cols, outs)
    r = Routes(g, T, E, topk, B, how)
    w = mrs.fp8_quantize(_rows(g, E * outs, cols, F32).view(E, outs, cols))
    ws = mrs.ProductWorkspace(T, E, topk, B, device=DEV)
    for per_route, weighted, kind in ((False, False, BF), (True, True, F32), (True, False, FH)):
        x = mrs.fp8_quantize(_rows(g, T * topk if per_route else T, cols, BF))
        out = torch.full((T * topk, outs), 7.0, dtype=kind, device=DEV)
        mrs.experts_product(x, w, *r.lists, sorted_weights=r.sw if weighted else None, out=out,
                            workspace=ws)
        assert ws.status_word() == 0
        want, size = _ref(x.codes.double() * x.scales.double()[:, None],
                          w.codes.double() * w.scales.double()[..., None], r)
        if weighted:
            by = r.weights.reshape(-1, 1).double()
            want, size = want * by, size * by
        routed = r.owners() >= 0
        _near(out[routed], want[routed], size[routed], cols, 4)
        _dropped_untouched(out, r, 7.0)


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("T,E,topk,cols,outs,B,how", SHAPES)
def test_grad_rows(T, E, topk, cols, outs, B, how, dtype):
    g = _gen("r", T, E, cols, outs)
    r = Routes(g, T, E, topk, B, how)
    w = _rows(g, E * outs, cols, dtype).view(E, outs, cols)
    ws = mrs.ProductWorkspace(T, E, topk, B, device=DEV)
    for per_route, kind in ((True, dtype), (False, F32)):
        grad = _rows(g, T * topk if per_route else T, outs, dtype)
        out = torch.full((T * topk, cols), 7.0, dtype=kind, device=DEV)
        mrs.experts_grad_rows(grad, w, *r.lists, out=out, workspace=ws)
        assert ws.status_word() == 0
        want, size = _ref(grad, w.transpose(1, 2), r)
        routed = r.owners() >= 0
        _near(out[routed], want[routed], size[routed], outs)
        _dropped_untouched(out, r, 7.0)


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("T,E,topk,cols,outs,B,how", SHAPES)
def test_grad_weights(T, E, topk, cols, outs, B, how, dtype):
    g = _gen("w", T, E, cols, outs)
    r = Routes(g, T, E, topk, B, how)
    ws = mrs.ProductWorkspace(T, E, topk, B, device=DEV)
    for gper, xper, kind in ((True, False, F32), (False, True, dtype)):
        grad = _rows(g, T * topk if gper else T, outs, dtype)
        x = _rows(g, T * topk if xper else T, cols, dtype)
        out = torch.full((E, outs, cols), 7.0, dtype=kind, device=DEV)
        mrs.experts_grad_weights(grad, x, E, *r.lists, out=out, workspace=ws)
        assert ws.status_word() == 0
        gd, xd, owner = _per_route(grad, r).double(), _per_route(x, r).double(), r.owners()
        for e in range(E):
            at = (owner == e).nonzero()[:, 0]
            want = gd[at].T @ xd[at]
            _near(out[e], want, gd[at].T.abs() @ xd[at].abs(), max(at.numel(), 1))
