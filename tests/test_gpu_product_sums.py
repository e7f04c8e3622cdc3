"""How near the experts' products and their gradients come to float64 over long contractions, on a
GB300, as a share of the results' norm.

Products of two bf16, fp16 or e4m3 values are exact in fp32.  An instruction of the tensor core adds 16
of them or more to an fp32 sum and cuts the result: the error of a cut is spread over a step, at most
2^-23 of the sum, 2^-23 / sqrt(3) in the mean square.  Of random terms the sum grows like the square
root of their number, two thirds of its last size on average: the cuts of n / 16 instructions come to
n / 16 * 2^-23 * 0.577 * 0.667 = 0.77 n / 16 * 2^-24 at most, if all have one sign.  Factors and an fp32
output add 2^-24 each.  The path for a few routes has eight sums of an eighth of the terms.

A lost step of 64 (or 128 in 8 bits) of n terms is sqrt(64 / n) of the norm, a lost row of n of a gradient
of weights sqrt(1 / n): both are far above the bound, which is tested with the mistake in the oracle.
"""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs
from test_gpu_products import BF, DEV, F32, FH, Routes, _gen, _per_route, _rows

pytestmark = pytest.mark.gpu

EIGHT = "e4m3"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


def _bound(n, few=False):
    return n / (128 if few else 16) * 2.0**-24 + 8 * 2.0**-24


def _far(got, want):
    """The distance as a share of the norm, on the CPU."""
    return ((got - want).norm() / want.norm()).item()


def _operands(g, T, E, outs, cols, kind):
    """(x, w for the call, x, w in float64)."""
    if kind == EIGHT:  # (made here: rows to 8 bits end at 16384 columns, those of the products later)
        def rows8(*lead):
            codes = (128 * torch.randn(*lead, cols, generator=g, device=DEV)).clamp(-448, 448)
            return mrs.Fp8Rows(codes.to(torch.float8_e4m3fn),
                               torch.rand(lead, generator=g, device=DEV) / 128 + 1e-3)

        x, w = rows8(T), rows8(E, outs)
        return x, w, *(q.codes.double() * q.scales.double()[..., None] for q in (x, w))
    x, w = _rows(g, T, cols, kind), _rows(g, E * outs, cols, kind).view(E, outs, cols)
    return x, w, x.double(), w.double()


# T, E: a few routes; narrow tiles; wide ones
@pytest.mark.parametrize("T,E", [(20, 3), (200, 8), (300, 2)])
@pytest.mark.parametrize("cols", [1040, 5136, 16384, 65536])
@pytest.mark.parametrize("kind", [BF, FH, EIGHT])
def test_product(kind, cols, T, E):
    g = _gen("sums", str(kind), cols, T)
    outs = 72
    r = Routes(g, T, E, 1, 16)
    x, w, xd, wd = _operands(g, T, E, outs, cols, kind)
    got = mrs.experts_product(x, w, *r.lists, dtype=F32).double().cpu()
    each = torch.stack([xd @ wd[e].T for e in range(E)])[r.owners(), torch.arange(T, device=DEV)].cpu()
    bound = _bound(cols, few=T <= 128)
    assert _far(got, each) <= bound
    deep = 128 if kind == EIGHT else 64
    step = slice(cols - deep, cols)  # the last one, as if it had been left out
    lost = torch.stack([xd[:, step] @ wd[e][:, step].T for e in range(E)])
    lost = lost[r.owners(), torch.arange(T, device=DEV)].cpu()
    assert _far(got, each - lost) > 10 * bound


@pytest.mark.parametrize("kind", [BF, EIGHT])
def test_product_of_many_rounds(kind):
    T, E, wide, cols = 3000, 2, 41416, 2080
    g = _gen("rounds", str(kind))
    r = Routes(g, T, E, 1, 64)
    x, w, xd, wd = _operands(g, T, E, wide, cols, kind)
    pick = torch.cat([torch.arange(300, device=DEV), torch.arange(wide - 300, wide, device=DEV)])
    got = mrs.experts_product(x, w, *r.lists, dtype=F32)[:, pick].double().cpu()
    each = torch.stack([xd @ wd[e][pick].T for e in range(E)])
    assert _far(got, each[r.owners(), torch.arange(T, device=DEV)].cpu()) <= _bound(cols)


@pytest.mark.parametrize("outs", [1032, 5128, 16384, 65536])
@pytest.mark.parametrize("T,E", [(20, 3), (200, 8), (300, 2)])
@pytest.mark.parametrize("kind", [BF, FH])
def test_gradient_of_rows(kind, T, E, outs):
    g = _gen("sums of rows", str(kind), outs, T)
    cols = 72
    r = Routes(g, T, E, 1, 16)
    grad, w = _rows(g, T, outs, kind), _rows(g, E * outs, cols, kind).view(E, outs, cols)
    got = mrs.experts_grad_rows(grad, w, *r.lists, dtype=F32).double().cpu()
    gd, at = grad.double(), (r.owners(), torch.arange(T, device=DEV))
    each = torch.stack([gd @ w[e].double() for e in range(E)])[at].cpu()
    lost = torch.stack([gd[:, -64:] @ w[e, -64:].double() for e in range(E)])[at].cpu()
    assert _far(got, each) <= _bound(outs)
    assert _far(got, each - lost) > 10 * _bound(outs)


@pytest.mark.parametrize("rows", [1000, 1025, 5000, 16384, 65537])
@pytest.mark.parametrize("kind", [BF, FH])
def test_gradient_of_weights(kind, rows):
    g = _gen("sums of weights", str(kind), rows)
    E, topk = 3, 2
    r = Routes(g, rows, E, topk, 16)
    x, grad = _rows(g, rows, 136, kind), _rows(g, rows * topk, 72, kind)
    got = mrs.experts_grad_weights(grad, x, E, *r.lists, dtype=F32).double().cpu()
    gd, xd, owner = grad.double(), _per_route(x, r).double(), r.owners()
    for e in range(E):
        at = (owner == e).nonzero()[:, 0]
        want, bound = (gd[at].T @ xd[at]).cpu(), _bound(at.numel())
        assert _far(got[e], want) <= bound
        for i in (0, at.numel() // 2, at.numel() - 1):  # one row of the run, as if it had been left out
            lost = torch.outer(gd[at[i]], xd[at[i]]).cpu()
            assert _far(got[e], want - lost) > 5 * bound
