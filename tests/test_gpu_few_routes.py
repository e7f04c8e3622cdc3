"""The products of a few routes give the same bits every call, on a GB300: a slot of weights is not filled
again before all of its readers have it.  Several groups of eight routes on the same expert take the same
weights one behind another, from L2, which is when the next copy of a slot is soonest there."""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs
from test_gpu_product_sums import EIGHT, _bound, _far, _operands
from test_gpu_products import BF, DEV, F32, FH, Routes, _gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


# T, E, topk, cols, outs
CASES = [(20, 1, 1, 8192, 264), (100, 1, 1, 8192, 2048), (128, 1, 1, 65536, 264), (64, 2, 1, 16384, 1024),
         (100, 4, 1, 3584, 768), (16, 8, 8, 7168, 2048), (1, 64, 16, 3584, 768), (9, 3, 2, 1040, 72)]


@pytest.mark.parametrize("T,E,topk,cols,outs", CASES)
@pytest.mark.parametrize("kind", [EIGHT, BF, FH])
def test_same_bits(kind, T, E, topk, cols, outs):
    g = _gen("few", T, E, cols)
    r = Routes(g, T, E, topk, 16)
    x, w, xd, wd = _operands(g, T, E, outs, cols, kind)
    ws = mrs.ProductWorkspace(T, E, topk, 16, device=DEV)
    first = mrs.experts_product(x, w, *r.lists, dtype=F32, workspace=ws)
    out = torch.empty_like(first)
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(300):
        out.fill_(7.0)
        mrs.experts_product(x, w, *r.lists, out=out, workspace=ws)
        differ += (out != first).sum()
    assert ws.status_word() == 0 and differ.item() == 0
    token, owner = torch.arange(T * topk, device=DEV) // topk, r.owners()
    want = torch.zeros(T * topk, outs, dtype=torch.float64, device=DEV)
    for e in range(E):
        at = (owner == e).nonzero()[:, 0]
        want[at] = xd[token[at]] @ wd[e].T
    assert _far(first.double().cpu(), want.cpu()) <= _bound(cols, few=True)
