"""Calls of the training and experts operators that their documentation allows beside the common
ones, on a GB300."""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


def _router(T, E, K, seed=0):
    g = torch.Generator().manual_seed(seed)
    logits = (1.5 * torch.randn(T, E, generator=g)).bfloat16()
    ids = torch.rand(T, E, generator=g).topk(K, dim=1).indices.int()
    return logits.to(DEV), ids.to(DEV)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,K", [(64, 6), (129, 5), (2056, 8)])
def test_the_loss_gradient_does_not_need_the_ids(E, K, softmax):
    # the same call with and without ids: the routes only steer the weights' term
    logits, ids = _router(200, E, K)
    counts = mrs.balance_loss(logits, ids, 0.5, softmax=softmax).counts
    term = dict(softmax=softmax, grad_loss=torch.ones(1, device=DEV), counts=counts, coef=0.5,
                dtype=torch.float32)
    want = mrs.route_backward(logits, ids, **term)
    assert torch.equal(mrs.route_backward(logits, None, topk=K, **term), want)
    assert want.any()
