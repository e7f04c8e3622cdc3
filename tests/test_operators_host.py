"""Host checks of the training and experts entry points: size queries and refusals, before any
device is touched (no GPU needed)."""
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


def _loss(lib, T=64, E=64, K=6, S=2, softmax=0, coef=0.1, x=BASE, ids=BASE + 0x10000,
          off=BASE + 0x20000, loss=BASE + 0x30000, counts=BASE + 0x40000, mean=BASE + 0x50000,
          ws=BASE + 0x100000, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = mrs.moe_balance_workspace_bytes(T, E, S) or 1 << 20
    return lib.moe_balance_loss(x, ids, off, T, E, K, S, softmax, coef, loss, counts, mean, ws,
                                ws_bytes, None)


def test_balance_loss_refuses(lib):
    assert _loss(lib, T=-1) == -6
    assert _loss(lib, E=0) == -2 and _loss(lib, E=4097) == -2
    assert _loss(lib, K=0) == -4 and _loss(lib, K=33) == -4 and _loss(lib, E=4, K=5) == -4
    assert _loss(lib, S=0) == -19 and _loss(lib, S=65537) == -19
    assert _loss(lib, off=None) == -19  # two sequences and no borders
    assert _loss(lib, T=(1 << 31) // 6 + 1) == -7
    assert _loss(lib, coef=NAN) == -11
    assert _loss(lib, ws=0) == -10 and _loss(lib, ws_bytes=64) == -10
    for name in ("x", "ids", "loss", "counts", "mean"):
        assert _loss(lib, **{name: 0}) == -1
    assert _loss(lib, x=BASE + 8) == -8 and _loss(lib, ws=BASE + 0x100004) == -8
    assert _loss(lib, counts=BASE + 0x40002) == -8
    assert _loss(lib, counts=BASE + 0x50010) == -9  # over the means
    assert _loss(lib, loss=BASE + 0x20004) == -9  # over the borders
    assert _loss(lib, mean=BASE + 64) == -9


def _backward(lib, T=64, E=64, K=6, S=1, softmax=0, R=2.5, coef=0.1, x=BASE, ids=BASE + 0x10000,
              gw=BASE + 0x20000, gl=BASE + 0x30000, counts=BASE + 0x40000, off=None,
              out=BASE + 0x50000, dt=0):
    return lib.moe_route_backward(x, ids, gw, gl, counts, off, T, E, K, S, softmax, R, coef, out,
                                  dt, None)


def test_route_backward_refuses(lib):
    assert _backward(lib, T=-1) == -6
    assert _backward(lib, E=5000) == -2
    assert _backward(lib, K=33) == -4
    assert _backward(lib, S=2) == -19
    assert _backward(lib, dt=1) == -17 and _backward(lib, dt=7) == -17
    assert _backward(lib, R=NAN) == -11 and _backward(lib, coef=float("inf")) == -11
    assert _backward(lib, x=0) == -1 and _backward(lib, out=0) == -1
    assert _backward(lib, ids=None) == -1  # with grad_weights
    assert _backward(lib, counts=None) == -1  # with grad_loss
    assert _backward(lib, out=BASE + 0x50008) == -8
    assert _backward(lib, gw=BASE + 0x20002) == -8
    assert _backward(lib, out=BASE + 16) == -9
    assert _backward(lib, counts=BASE + 0x50010) == -9
    assert _backward(lib, T=0) == 0


def test_mxfp4_sizes_and_refusals(lib):
    assert [mrs.moe_mxfp4_scale_cols(c) for c in (32, 128, 160, 3584, 32768)] == [4, 4, 8, 112, 1024]
    assert [mrs.moe_mxfp4_scale_cols(c) for c in (0, -32, 33, 16, 32800)] == [0] * 5

    def q(x=BASE, dt=0, rows=8, cols=64, stride=64, codes=BASE + 0x10000, scales=BASE + 0x20000):
        return lib.moe_mxfp4_quantize(x, dt, rows, cols, stride, codes, scales, None)

    def d(codes=BASE + 0x10000, scales=BASE + 0x20000, rows=8, cols=64, y=BASE, dt=0, stride=64):
        return lib.moe_mxfp4_dequantize(codes, scales, rows, cols, y, dt, stride, None)

    for f in (q, d):
        assert f(rows=-1) == -20
        assert f(cols=48) == -18 and f(cols=0) == -18 and f(cols=32800, stride=32800) == -18
        assert f(stride=56) == -18
        assert f(rows=1 << 41) == -7
        assert f(codes=0) == -1 and f(scales=0) == -1
        assert f(codes=BASE + 0x10008) == -8 and f(scales=BASE + 0x20002) == -8
        assert f(stride=68) == -8
        assert f(rows=0) == 0
    assert q(dt=3) == -17 and d(dt=1) == -17
    assert q(x=0) == -1 and d(y=0) == -1
    assert q(x=BASE + 2) == -8 and d(y=BASE + 4) == -8
    assert q(codes=BASE + 1008) == -9 and q(scales=BASE + 0x10080) == -9
    assert d(y=BASE + 0x10000 - 16) == -9


def _experts(lib, T=8, E=4, K=2, cols=64, N=16, B=16, per=0, xc=BASE, xs=BASE + 0x1000,
             wc=BASE + 0x2000, ws=BASE + 0x4000, sid=BASE + 0x6000, sw=BASE + 0x8000,
             eid=BASE + 0xA000, npp=BASE + 0xB000, out=BASE + 0x10000, dt=0, work=BASE + 0x40000,
             work_bytes=256):
    return lib.moe_experts_mxfp4(xc, xs, per, wc, ws, T, E, K, cols, N, B, sid, sw, eid, npp, out,
                                 dt, work, work_bytes, None)


def test_experts_refuse(lib):
    assert mrs.moe_experts_mxfp4_workspace_bytes(8, 4, 2, 16) % 16 == 0
    assert mrs.moe_experts_mxfp4_workspace_bytes(8, 4, 2, 12) == 0
    assert _experts(lib, T=-1) == -6
    assert _experts(lib, E=0) == -2 and _experts(lib, E=4097) == -2
    assert _experts(lib, K=0) == -4 and _experts(lib, K=33) == -4
    assert _experts(lib, B=24) == -5 and _experts(lib, B=2048) == -5
    assert _experts(lib, cols=48) == -18 and _experts(lib, N=12) == -18 and _experts(lib, N=0) == -18
    assert _experts(lib, N=65544) == -18
    assert _experts(lib, dt=1) == -17
    assert _experts(lib, T=1 << 30, K=4) == -7
    assert _experts(lib, work=0) == -10 and _experts(lib, work_bytes=128) == -10
    for name in ("xc", "xs", "wc", "ws", "sid", "eid", "npp", "out"):
        assert _experts(lib, **{name: 0}) == -1
    assert _experts(lib, xc=BASE + 8) == -8 and _experts(lib, ws=BASE + 0x4002) == -8
    assert _experts(lib, out=BASE + 0x10008) == -8
    assert _experts(lib, out=BASE + 0x2000) == -9
    assert _experts(lib, work=BASE + 0x10010) == -9
    assert _experts(lib, T=0) == 0


def test_status_texts(lib):
    for code in range(-20, 1):
        assert mrs.strerror(code) != "unknown status"


def test_binding_refuses_host_and_misshaped_buffers():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mrs.moe_balance_loss(x, ids, None, False, 0.1, x, ids, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        mrs.moe_route_backward(x, ids, None, None, None, None, False, 1.0, 0.1, x)
    with pytest.raises(ValueError, match="CUDA"):
        mrs.moe_mxfp4_quantize(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        mrs.moe_mxfp4_dequantize(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        mrs.moe_experts_mxfp4(x, x, x, x, 4, 2, 16, ids, None, ids, ids, x, x)
    with pytest.raises(ValueError, match="multiple of 32"):
        mrs.Mxfp4Rows.allocate(4, 40, device="cpu")
    with pytest.raises(ValueError):
        mrs.BalanceBuffers.allocate(4, 0, device="cpu")


def _packed(lib, op, n, *values):
    import struct

    fmt = "=qq" + "".join("d" if isinstance(v, float) else "q" for v in values)
    return lib.moe_call_packed(struct.pack(fmt, op, n, *values))


def test_packed_calls_reach_their_operations(lib):
    # every operation's first refusals, and the counts of arguments
    assert _packed(lib, 0, 0) == -21 and _packed(lib, 6, 0) == -21
    for op in (1, 2, 3, 4, 5):
        assert _packed(lib, op, 7) == -21
    b = BASE
    loss = [b, b, 0, -1, 64, 6, 1, 0, 0.5, b, b, b, b, 1 << 20, 0]
    assert _packed(lib, 1, 15, *loss) == -6
    loss[3], loss[4] = 4, 5000
    assert _packed(lib, 1, 15, *loss) == -2
    loss[4], loss[8] = 64, NAN
    assert _packed(lib, 1, 15, *loss) == -11
    loss[3] = 1 << 40  # does not fit the argument's type
    assert _packed(lib, 1, 15, *loss) == -7
    back = [b, b, b, b, b, 0, 4, 64, 6, 1, 0, 2.5, 0.1, b + 0x10000, 9, 0]
    assert _packed(lib, 2, 16, *back) == -17
    back[14], back[12] = 0, float("inf")
    assert _packed(lib, 2, 16, *back) == -11
    assert _packed(lib, 3, 8, b, 0, 8, 48, 48, b, b, 0) == -18
    assert _packed(lib, 3, 8, b, 0, 1 << 41, 64, 64, b, b, 0) == -7
    assert _packed(lib, 4, 8, b, b, -1, 64, b, 0, 64, 0) == -20
    ex = [b, b, 0, b, b, 8, 4, 2, 64, 16, 24, b, b, b, b, b, 0, b, 256, 0]
    assert _packed(lib, 5, 20, *ex) == -5
    ex[10], ex[18] = 16, 8
    assert _packed(lib, 5, 20, *ex) == -10
    assert lib.moe_call_packed(None) == -1
    assert mrs.strerror(-21) != "unknown status"
