"""Tensors of the wrong number of dimensions are refused as such, before buffers are made for them."""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


@pytest.mark.parametrize("shape", [(), (64,), (2, 4, 64)])
def test_norm_gradient(shape):
    s = torch.zeros(shape, dtype=BF, device=DEV)
    gain, rstd = torch.ones(64, dtype=BF, device=DEV), torch.ones(8, device=DEV)
    with pytest.raises(ValueError, match="s must be .T, cols"):
        mrs.rms_norm_backward(s, gain, rstd, s)


@pytest.mark.parametrize("shape", [(), (64,), (16, 64), (1, 2, 16, 64)])
def test_weights(shape):
    i = torch.zeros(64, dtype=torch.int32, device=DEV)
    lists = (4, 2, 16, i, i, i)
    x = torch.zeros(4, 64, dtype=BF, device=DEV)
    grad = torch.zeros(8, 16, dtype=BF, device=DEV)
    w = torch.zeros(shape, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="w must be .E, outs, cols"):
        mrs.experts_product(x, w, *lists)
    with pytest.raises(ValueError, match="w must be .E, outs, cols"):
        mrs.experts_grad_rows(grad, w, *lists)
    with pytest.raises(ValueError, match="must be .E, outs, cols|of 2 experts"):
        mrs.experts_grad_weights(grad, x, 2, *lists, out=w)
    if len(shape) > 1:
        with pytest.raises(ValueError, match="E, outs, cols"):
            mrs.experts_product(mrs.fp8_quantize(x), mrs.fp8_quantize(w[:1]), *lists)
    if len(shape) != 2:
        with pytest.raises(ValueError, match="must be matrices"):
            mrs.experts_grad_weights(w, x, 2, *lists)
        with pytest.raises(ValueError, match="must be matrices"):
            mrs.experts_grad_weights(grad, w, 2, *lists)
