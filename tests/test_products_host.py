"""Host checks of the experts' products in 16 and 8 bits and their gradients: sizes and refusals, before
any device is touched (no GPU needed)."""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs
from moe_expert_routing_sort_gb300 import _build

B = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mrs.load()


def _product(lib, T=8, E=4, K=2, cols=64, outs=16, bm=16, x=B, dt=0, xs=0, per=0, w=B + 0x10000, ws=0,
             sid=B + 0x20000, sw=B + 0x21000, eid=B + 0x22000, npp=B + 0x23000, out=B + 0x30000,
             odt=0, work=B + 0x100000, work_bytes=1 << 20):
    return lib.moe_experts_product(x, dt, xs, per, w, ws, T, E, K, cols, outs, bm, sid, sw, eid, npp,
                                   out, odt, work, work_bytes, None)


def _rows(lib, T=8, E=4, K=2, cols=64, outs=16, bm=16, g=B, dt=0, per=1, w=B + 0x10000,
          sid=B + 0x20000, eid=B + 0x22000, npp=B + 0x23000, out=B + 0x30000, odt=0,
          work=B + 0x100000, work_bytes=1 << 20):
    return lib.moe_experts_grad_rows(g, dt, per, w, T, E, K, cols, outs, bm, sid, eid, npp, out, odt,
                                     work, work_bytes, None)


def _weights(lib, T=8, E=4, K=2, cols=64, outs=16, bm=16, g=B, dt=0, gper=1, x=B + 0x10000, xper=0,
             sid=B + 0x20000, eid=B + 0x22000, npp=B + 0x23000, out=B + 0x30000, odt=2,
             work=B + 0x100000, work_bytes=1 << 20):
    return lib.moe_experts_grad_weights(g, dt, gper, x, xper, T, E, K, cols, outs, bm, sid, eid, npp,
                                        out, odt, work, work_bytes, None)


def test_workspace_sizes(lib):
    size = mrs.moe_experts_product_workspace_bytes
    assert size(8, 4, 2, 16) % 16 == 0 and size(8, 4, 2, 16) >= 256
    assert size(8192, 896, 16, 128) > size(512, 896, 16, 128)
    for bad in ((-1, 4, 2, 16), (8, 0, 2, 16), (8, 4097, 2, 16), (8, 4, 0, 16), (8, 4, 33, 16),
                (8, 4, 2, 12), (8, 4, 2, 2048), (1 << 30, 4, 4, 16), (1 << 27, 4, 16, 1024)):
        assert size(*bad) == 0
    with pytest.raises(ValueError, match="invalid shape"):
        mrs.ProductWorkspace.allocate(8, 4, 2, 24, device="cpu")


@pytest.mark.parametrize("call", [_product, _rows, _weights])
def test_shapes_are_refused(lib, call):
    assert call(lib, T=-1) == -6
    assert call(lib, E=0) == -2 and call(lib, E=4097) == -2
    assert call(lib, K=0) == -4 and call(lib, K=33) == -4
    assert call(lib, bm=24) == -5 and call(lib, bm=0) == -5 and call(lib, bm=2048) == -5
    assert call(lib, cols=60) == -18 and call(lib, cols=0) == -18 and call(lib, cols=65544) == -18
    assert call(lib, outs=12) == -18 and call(lib, outs=0) == -18 and call(lib, outs=65544) == -18
    assert call(lib, dt=2) == -17 and call(lib, dt=5) == -17 and call(lib, odt=3) == -17
    assert call(lib, T=1 << 30, K=4) == -7 and call(lib, T=1 << 27, K=16, bm=1024) == -7
    assert call(lib, work=0) == -10 and call(lib, work_bytes=64) == -10
    for name in ("sid", "eid", "npp", "out"):
        assert call(lib, **{name: 0}) == -1
    assert call(lib, out=B + 0x30008) == -8 and call(lib, sid=B + 0x20002) == -8
    assert call(lib, work=B + 0x100008) == -8
    assert call(lib, out=B + 16) == -9 and call(lib, work=B + 0x30010) == -9


def test_product_is_refused(lib):
    assert _product(lib, T=0) == 0
    assert _product(lib, x=0) == -1 and _product(lib, w=0) == -1
    assert _product(lib, x=B + 8) == -8 and _product(lib, w=B + 0x10008) == -8
    assert _product(lib, sw=B + 0x21002) == -8
    # 8 bits: both scales, rows of multiples of 16; 16 bits: none
    assert _product(lib, dt=3) == -1
    assert _product(lib, dt=3, xs=B + 0x40000, ws=0) == -1
    assert _product(lib, dt=3, xs=B + 0x40000, ws=B + 0x50000, cols=72) == -18
    assert _product(lib, dt=3, xs=B + 0x40002, ws=B + 0x50000) == -8
    assert _product(lib, dt=3, xs=B + 0x30010, ws=B + 0x50000) == -9
    assert _product(lib, xs=B + 0x40000) == -17
    assert _product(lib, out=B + 0x21010) == -9


def test_gradients_are_refused(lib):
    assert _rows(lib, T=0) == 0
    assert _rows(lib, dt=3) == -17 and _rows(lib, g=0) == -1 and _rows(lib, w=0) == -1
    assert _weights(lib, dt=3) == -17 and _weights(lib, dt=0, odt=1) == -17
    assert _weights(lib, g=0) == -1 and _weights(lib, x=0) == -1
    assert _weights(lib, T=0, out=0) == -1  # zeros have to go somewhere
    assert _weights(lib, x=B + 0x10004) == -8 and _weights(lib, out=B + 0x10000) == -9


def test_packed_calls(lib):
    # the numbers of arguments that the operations take, and values outside an integer's type
    import struct

    def call(op, n, *args):
        return lib.moe_call_packed(struct.pack(f"=qq{len(args)}q", op, n, *args))

    for op, n in ((6, 8), (7, 17), (8, 16), (9, 10), (10, 10), (11, 21), (12, 18), (13, 19)):
        assert call(op, n + 1, *([0] * (n + 1))) == -21
        assert call(op, n - 1, *([0] * (n - 1))) == -21
    assert call(6, 8, B, 1 << 40, 8, 64, 64, B, B, 0) == -7
    assert call(14, 8, *([0] * 8)) == -21


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 16, 64, dtype=torch.bfloat16)
    ids = torch.zeros(64, dtype=torch.int32)
    for call in (lambda: mrs.experts_product(x, w, 4, 1, 16, ids, ids, ids),
                 lambda: mrs.experts_grad_rows(x, w, 4, 1, 16, ids, ids, ids),
                 lambda: mrs.experts_grad_weights(x, x, 2, 4, 1, 16, ids, ids, ids)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
