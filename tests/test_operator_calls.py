"""What the bindings of the training and experts operators make of a call's arguments (no GPU)."""
import os
import subprocess
import sys

import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs
from _shapes import STAYING, plan_row
from moe_expert_routing_sort_gb300 import _build, training


@pytest.fixture
def backward_args(monkeypatch):
    """The arguments that reach the C entry of the gradient, on host tensors."""
    seen = []
    monkeypatch.setattr(training, "cuda_device", lambda t, name: 0)
    monkeypatch.setattr(training, "need", lambda t, dtype, numel, dev, name: name)
    monkeypatch.setattr(training, "_backward", lambda dev, stream, *args: seen.append(args))
    return seen


def test_a_loss_gradient_without_ids_has_its_routes_per_token(backward_args):
    T, E, K = 8, 16, 6
    x = torch.zeros(T, E, dtype=torch.bfloat16)
    ids = torch.zeros(T, K, dtype=torch.int32)
    loss = dict(grad_loss=torch.ones(1), counts=torch.zeros(1, E, dtype=torch.int32), coef=0.5)
    training.route_backward(x, ids, **loss)
    training.route_backward(x, ids, topk=K, **loss)
    training.route_backward(x, None, topk=K, **loss)
    training.moe_route_backward(x, None, None, loss["grad_loss"], loss["counts"], None, False, 1.0,
                                0.5, torch.zeros(T, E), topk=K)
    at = 8  # logits, ids, weights, loss, counts, offsets, T, E, topk
    assert [a[at] for a in backward_args] == [K] * 4
    with pytest.raises(ValueError, match="needs topk"):
        training.route_backward(x, None, **loss)
    with pytest.raises(ValueError, match="6 routes per token"):
        training.route_backward(x, ids, topk=4, **loss)
    training.route_backward(x, None)  # no term at all: zeros, whatever topk
    assert len(backward_args) == 5


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mrs.load()


def test_experts_without_a_workspace_take_the_librarys_word(lib):
    b = 0x7F0000000000

    def call(T, work, work_bytes, codes=0):
        return lib.moe_experts_mxfp4(codes, b, 0, b, b, T, 4, 2, 64, 16, 16, b, None, b, b, b, 0,
                                     work, work_bytes, None)

    assert call(8, None, 0) == -1  # past the workspace's check: the codes are missing
    assert call(0, None, 0) == 0
    assert call(8, None, 256) == -10 and call(8, b, 0) == -10 and call(8, b, 128) == -10
    assert lib.moe_experts_mxfp4_status(None, 0, None) == -1
    assert lib.moe_experts_mxfp4_status(b + 2, 0, None) == -8
    with pytest.raises(ValueError, match="CUDA"):
        mrs.moe_experts_mxfp4_status(torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="invalid shape"):
        mrs.ExpertsWorkspace.allocate(8, 4, 2, 24, device="cpu")
    assert mrs.ExpertsWorkspace.allocate(8, 4, 2, 16, device="cpu").tensor.numel() >= 4
    assert (mrs.DEVICE_BAD_EXPERT_ID, mrs.DEVICE_WAIT_TIMEOUT) == (1, 2)


def test_the_package_imports_without_cuda_in_torch():
    # size queries, host checks and the build ask nothing of torch's CUDA side
    code = ("import torch\n"
            "del torch._C._cuda_getCurrentRawStream\n"
            "import moe_expert_routing_sort_gb300 as mrs\n"
            "assert mrs.moe_mxfp4_scale_cols(160) == 8\n"
            "assert mrs.moe_balance_workspace_bytes(8, 64, 1) > 0\n")
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert got.returncode == 0, got.stderr


@pytest.mark.parametrize("shape,row", [(s, tuple(r)) for s, *r in STAYING])
def test_shapes_whose_rows_stay_for_several_tiles(lib, shape, row):
    plan = mrs.moe_experts_mxfp4_plan(*shape, sms=152)
    assert plan.unit_tiles > 1 and plan_row(plan, shape[4]) == row
    assert plan.units == -(-plan.tiles // plan.unit_tiles) and plan.steps == -(-shape[3] // 256)


def test_plans_of_other_calls(lib):
    plan = mrs.moe_experts_mxfp4_plan
    # one token: a block an expert, nothing stays; few wide experts: tiles of 256, which do not stay
    assert plan(1, 896, 16, 3584, 768, 16) == (96, 1, 1, 8, 1, 8, 14)
    assert plan(8192, 64, 8, 7168, 2048, 128) == (256, 1, 1, 8, 1, 8, 28)
    assert plan(8192, 896, 16, 384, 3584, 128).unit_tiles == 19
    assert any(s[2] and s[0] == 192 for _, *s in STAYING)
    for bad in [(0, 4, 2, 64, 16, 16), (8, 0, 2, 64, 16, 16), (8, 4, 0, 64, 16, 16),
                (8, 4, 2, 48, 16, 16), (8, 4, 2, 64, 12, 16), (8, 4, 2, 64, 16, 24),
                (1 << 30, 4, 4, 64, 16, 16)]:
        with pytest.raises(mrs.RouteSortError):
            plan(*bad)
    with pytest.raises(mrs.RouteSortError):
        plan(8, 4, 2, 64, 16, 16, sms=0)
    assert lib.moe_experts_mxfp4_plan(8, 4, 2, 64, 16, 16, 152, None) == -1
