"""What the bindings of the training and experts operators make of a call's arguments (no GPU)."""
import pytest
import torch

from moe_expert_routing_sort_gb300 import training


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
