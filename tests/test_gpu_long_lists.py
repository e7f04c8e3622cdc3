"""The experts' products over lists as long as their documentation allows, on a GB300.

Values are small whole numbers in a few tokens and zeros in the others, so that every sum is a whole
number below 2^24: exact in fp32 and in the tensor core's sums.  One lost or repeated row shows.
"""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _one_expert(T, topk, B):
    """The sorted list of T * topk routes of one expert."""
    n = T * topk
    P = mrs.moe_sort_max_padded(T, 1, topk, B)
    sid = torch.arange(P, dtype=torch.int32, device=DEV).clamp_(max=n)
    eid = torch.zeros(P // B, dtype=torch.int32, device=DEV)
    npp = torch.full((1,), (n + B - 1) // B * B, dtype=torch.int32, device=DEV)
    return T, topk, B, sid, eid, npp


def _few_rows(T, cols, seed):
    """[T, cols] of zeros but for the first and last 50 tokens and some 1000 in between, which hold
    whole numbers from -2 to 2."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    at = torch.cat([torch.arange(50, device=DEV), torch.arange(T - 50, T, device=DEV),
                    torch.randint(50, T - 50, (1000,), generator=g, device=DEV)]).unique()
    x = torch.zeros(T, cols, dtype=BF, device=DEV)
    x[at] = torch.randint(-2, 3, (at.numel(), cols), generator=g, device=DEV).to(BF)
    return x, at


def _check_grad_weights(lists, dtype, seed):
    T, topk = lists[:2]
    x, at = _few_rows(T, 16, seed)
    grad = torch.ones(T, 8, dtype=BF, device=DEV)
    grad[at] = torch.randint(-2, 3, (at.numel(), 8), device=DEV).to(BF)
    ws = mrs.ProductWorkspace(T, 1, topk, lists[2], device=DEV)
    dw = mrs.experts_grad_weights(grad, x, 1, *lists, dtype=dtype, workspace=ws)
    assert ws.status_word() == 0
    want = topk * (grad[at].double().T @ x[at].double())
    assert torch.equal(dw[0], want.to(dtype))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_gradient_of_weights_of_an_expert_of_134_million_rows(dtype):
    # two million steps of one tile: the waits for it last as long
    _check_grad_weights(_one_expert(1 << 22, 32, 128), dtype, 1)


# 2^31 - 2 routes in blocks of one row: what is counted ahead of the last row, and past the last block,
# does not fit 31 bits
LONGEST = (69273666, 31, 1)


def test_products_of_the_longest_list():
    T, topk, B = LONGEST
    lists = _one_expert(T, topk, B)
    x, at = _few_rows(T, 8, 2)
    g = torch.Generator(device=DEV).manual_seed(3)
    w = torch.randint(-2, 3, (1, 8, 8), generator=g, device=DEV).to(BF)
    ws = mrs.ProductWorkspace(T, 1, topk, B, device=DEV)
    out = torch.empty(T * topk, 8, dtype=BF, device=DEV)
    for call, by in ((mrs.experts_product, w[0].T), (mrs.experts_grad_rows, w[0])):
        out.fill_(7.0)
        call(x, w, *lists, out=out, workspace=ws)
        assert ws.status_word() == 0
        want = (x.float() @ by.float()).to(BF)
        each = out.view(T, topk, 8)
        for i in range(0, T, 1 << 22):
            assert (each[i:i + (1 << 22)] == want[i:i + (1 << 22), None]).all()


def test_gradient_of_weights_of_the_longest_list():
    _check_grad_weights(_one_expert(*LONGEST), F32, 4)
