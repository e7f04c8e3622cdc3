"""Experts' products whose rows stay in shared memory for several output tiles, on a GB300, against
the same float64 implementation and tolerances as their other tests.  (Some shapes of
test_product_many_tiles say that of themselves and were planned otherwise later; these ask the
plan.)"""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs
from _shapes import STAYING, plan_row
from test_gpu_experts import _check_product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape,row", [(s, tuple(r)) for s, *r in STAYING])
def test_rows_that_stay_for_several_tiles(shape, row, dtype):
    T, E, K, cols, N, B = shape
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    plan = mrs.moe_experts_mxfp4_plan(*shape, sms=sms)
    assert plan.unit_tiles > 1 and plan_row(plan, N) == row
    wide = dtype == torch.float32
    _check_product(T, E, K, cols, N, B, dtype=dtype, per_route=wide, weighted=wide,
                   dist="uniform" if wide else "drops")
