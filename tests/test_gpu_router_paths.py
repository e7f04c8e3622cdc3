"""Paths of the router training kernels that take large or particular shapes, on a GB300, against the
same float64 implementations and tolerances as their other tests: rings of rows that come round, every
width of a router's row, counts beyond those loaded ahead."""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs
from test_gpu_training import REL, _check_grad, _check_loss, _inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


# E, K: 16 columns a lane in vectors, and two warps a row
WIDTHS = [(264, 8), (384, 6), (512, 16), (1032, 4), (1536, 8), (2048, 8)]


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("T", [1, 67, 1000])
@pytest.mark.parametrize("E,K", WIDTHS)
def test_loss_of_router_widths(E, K, T, softmax):
    logits, ids = _inputs(T, E, K, seed=E + T)
    _check_loss(logits, ids, None, 0.01, softmax)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("T", [1, 700])
@pytest.mark.parametrize("E,K", WIDTHS)
def test_gradient_of_router_widths(E, K, T, softmax, dtype):
    logits, ids = _inputs(T, E, K, seed=E + T)
    _check_grad(logits, ids, None, softmax, dtype)


# More than four rows a group of warps and stretch at 152 SMs, for each number of warps a row: a
# lane's four slots are filled again.  Groups of a CTA: 16, 16, 8, 5 and 4.
LONG = [(128, 6, 24000), (896, 16, 12000), (1536, 8, 9000), (2504, 4, 5000), (4096, 8, 4000)]


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,K,T", LONG)
def test_rings_that_come_round(E, K, T, softmax):
    logits, ids = _inputs(T, E, K, seed=E)
    # one sequence, and borders that cut the CTAs' ranges, so that rings are opened again
    for off in (None, [3, T // 3, T // 3 + 7, T // 2, T - 5]):
        _check_loss(logits, ids, off, 0.1, softmax)
        _check_grad(logits, ids, off, softmax, torch.float32)
    _check_grad(logits, ids, None, softmax, torch.bfloat16)


@pytest.mark.parametrize("E", [64, 129])
def test_more_routes_than_are_loaded_ahead(E):
    # 108 tokens a CTA with 32 routes each, 2048 of which are loaded ahead of the rows
    T, K = 16384, 32
    logits, ids = _inputs(T, E, K, seed=E)
    _check_loss(logits, ids, None, 0.1, False)
    _check_loss(logits, ids, [0, 100, 16000], 0.1, True)


def test_gradients_of_the_softmax_weights_match_the_route_step():
    # the weights that moe_route_sort_softmax returns are those the gradient is taken of
    T, E, K, R = 64, 256, 8, 2.5
    logits, _ = _inputs(T, E, K, drop=False)
    out = mrs.route_sort_softmax(logits, K, R, 16)
    x = logits.double().cpu().requires_grad_()
    u = torch.softmax(x, 1).gather(1, out.topk_ids.long().cpu())
    w = R * u / u.sum(1, keepdim=True)
    assert (w.detach() - out.topk_weights.double().cpu()).abs().max() <= 1e-6
    gw = torch.randn(T, K, generator=torch.Generator().manual_seed(2))
    ref = torch.autograd.grad((w * gw).sum(), x)[0]
    got = mrs.route_backward(logits, out.topk_ids, gw.to(DEV), R, softmax=True, dtype=torch.float32)
    assert (got.double().cpu() - ref).abs().max() <= REL * R * gw.abs().max()
