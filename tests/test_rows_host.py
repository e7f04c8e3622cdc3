"""Host checks of the operators on rows (norm, gated activation, rows in 8 bits): refusals, before
any device is touched (no GPU needed)."""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs
from moe_expert_routing_sort_gb300 import _build

BASE = 0x7F0000000000
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mrs.load()


def test_quantize_refuses(lib):
    def q(x=BASE, dt=0, rows=8, cols=64, stride=64, codes=BASE + 0x10000, scales=BASE + 0x20000):
        return lib.moe_fp8_quantize(x, dt, rows, cols, stride, codes, scales, None)

    assert q(dt=3) == -17 and q(dt=-1) == -17
    assert q(rows=-1) == -20 and q(rows=1 << 31) == -7
    assert q(cols=60, stride=64) == -18 and q(cols=0) == -18 and q(cols=16392, stride=16392) == -18
    assert q(stride=56) == -18
    assert q(rows=0) == 0
    assert q(x=0) == -1 and q(codes=0) == -1 and q(scales=0) == -1
    assert q(x=BASE + 8) == -8 and q(stride=68) == -8 and q(codes=BASE + 0x10004) == -8
    assert q(scales=BASE + 0x20002) == -8
    assert q(codes=BASE + 1016) == -9 and q(scales=BASE + 0x10008) == -9


def _norm(lib, x=BASE, dt=0, stride=64, parts=2, res=BASE + 0x10000, rstride=64, rows=8, cols=64,
          gain=BASE + 0x20000, gdt=0, eps=1e-6, y=BASE + 0x30000, s=BASE + 0x40000,
          codes=BASE + 0x50000, scales=BASE + 0x60000, rstd=BASE + 0x70000):
    return lib.moe_rms_norm(x, dt, stride, parts, res, rstride, rows, cols, gain, gdt, eps, y, s,
                            codes, scales, rstd, None)


def test_norm_refuses(lib):
    assert _norm(lib, dt=2) == -17 and _norm(lib, gdt=1) == -17 and _norm(lib, gdt=3) == -17
    assert _norm(lib, rows=-1) == -20 and _norm(lib, rows=1 << 31) == -7
    assert _norm(lib, parts=0) == -4 and _norm(lib, parts=33) == -4
    assert _norm(lib, cols=68, stride=72, rstride=72) == -18 and _norm(lib, stride=56) == -18
    assert _norm(lib, rstride=56) == -18
    assert _norm(lib, eps=-1.0) == -11 and _norm(lib, eps=NAN) == -11
    assert _norm(lib, rows=0) == 0
    assert _norm(lib, x=0) == -1 and _norm(lib, gain=0) == -1
    assert _norm(lib, y=0, s=0, codes=0, scales=0, rstd=0) == -1
    assert _norm(lib, codes=0) == -1 and _norm(lib, scales=0) == -1
    for name in ("x", "res", "gain", "y", "s"):
        at = {"x": 0, "res": 0x10000, "gain": 0x20000, "y": 0x30000, "s": 0x40000}[name]
        assert _norm(lib, **{name: BASE + at + 8}) == -8
    assert _norm(lib, stride=68) == -8 and _norm(lib, rstride=68) == -8
    assert _norm(lib, y=BASE + 64) == -9 and _norm(lib, y=BASE + 0x40010) == -9
    assert _norm(lib, s=BASE + 0x10010) == -9  # over the residual, but not in its place
    assert _norm(lib, s=BASE + 0x10000, rstride=72) == -9  # nor with rows further apart


def _norm_grad(lib, s=BASE, dt=0, gain=BASE + 0x10000, gdt=0, rstd=BASE + 0x20000,
               grad=BASE + 0x30000, rows_=BASE + 0x40000, parts=2, gsum=BASE + 0x50000, rows=8,
               cols=64, gx=BASE + 0x60000, gg=BASE + 0x70000, ws=BASE + 0x1000000, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = mrs.moe_rms_norm_backward_workspace_bytes(cols) or 1 << 20
    return lib.moe_rms_norm_backward(s, dt, gain, gdt, rstd, grad, rows_, parts, gsum, rows, cols,
                                     gx, gg, ws, ws_bytes, None)


def test_norm_backward_refuses(lib):
    assert mrs.moe_rms_norm_backward_workspace_bytes(64) % 16 == 0
    assert [mrs.moe_rms_norm_backward_workspace_bytes(c) for c in (0, 4, 12, 16392)] == [0] * 4
    assert _norm_grad(lib, dt=2) == -17 and _norm_grad(lib, gdt=1) == -17
    assert _norm_grad(lib, rows=-1) == -20 and _norm_grad(lib, parts=0) == -4
    assert _norm_grad(lib, cols=20) == -18 and _norm_grad(lib, rows=1 << 31) == -7
    assert _norm_grad(lib, ws=0) == -10 and _norm_grad(lib, ws_bytes=64) == -10
    for name in ("s", "gain", "rstd", "gx"):
        assert _norm_grad(lib, **{name: 0}) == -1
    assert _norm_grad(lib, grad=0, rows_=0) == -1
    assert _norm_grad(lib, gx=BASE + 0x60008) == -8 and _norm_grad(lib, gg=BASE + 0x70002) == -8
    assert _norm_grad(lib, gx=BASE + 0x50000) == -9  # the gradient of the sum stays as it is
    assert _norm_grad(lib, ws=BASE + 0x40010) == -9
    assert _norm_grad(lib, rows=0, gg=0, ws=0) == 0


def _gated(lib, x=BASE, dt=0, stride=128, rows=8, cols=64, w=BASE + 0x10000, y=BASE + 0x20000,
           codes=BASE + 0x30000, scales=BASE + 0x40000):
    return lib.moe_swiglu(x, dt, stride, rows, cols, w, y, codes, scales, None)


def _gated_grad(lib, g=BASE, x=BASE + 0x10000, dt=0, stride=128, rows=8, cols=64, w=BASE + 0x20000,
                gx=BASE + 0x30000, gw=BASE + 0x40000):
    return lib.moe_swiglu_backward(g, x, dt, stride, rows, cols, w, gx, gw, None)


def test_swiglu_refuses(lib):
    for f in (_gated, _gated_grad):
        assert f(lib, dt=2) == -17 and f(lib, rows=-1) == -20 and f(lib, rows=1 << 31) == -7
        assert f(lib, cols=60) == -18 and f(lib, stride=120) == -18 and f(lib, x=0) == -1
        assert f(lib, stride=132) == -8 and f(lib, rows=0) == 0
    assert _gated(lib, x=BASE + 2) == -8 and _gated(lib, w=BASE + 0x10002) == -8
    assert _gated(lib, y=0, codes=0, scales=0) == -1 and _gated(lib, codes=0) == -1
    assert _gated(lib, y=BASE + 64) == -9 and _gated(lib, codes=BASE + 0x20008) == -9
    assert _gated_grad(lib, g=0) == -1 and _gated_grad(lib, gx=0) == -1
    assert _gated_grad(lib, gx=BASE + 0x10000) == -9 and _gated_grad(lib, gw=BASE + 0x30004) == -9
    assert _gated_grad(lib, g=BASE + 8) == -8


def test_python_refuses_host_tensors():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    for call in (lambda: mrs.rms_norm(x, w), lambda: mrs.swiglu(x), lambda: mrs.fp8_quantize(x),
                 lambda: mrs.swiglu_backward(x, x), lambda: mrs.rms_norm_backward(x, w, x, x),
                 lambda: mrs.Fp8Rows.allocate(4, 64, device="cpu")):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="needs an output"):
        mrs.NormBuffers.allocate(4, 64, y=False, device="cpu")
