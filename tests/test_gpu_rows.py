"""Norm, gated activation, their gradients and rows in 8 bits on a GB300, against plain float64
implementations.

Tolerances, u = 2^-24 (half a step of fp32, relative):
* fp32 sums of n terms in any order of at most 64 levels here: 64 u sum |terms| (a thread adds up to
  16 terms, then at most 5 + 32 levels of shuffles and warps).
* 16-bit outputs: half a step of the type (2^-8, 2^-11) plus the fp32 error ahead of it; where that
  is near a border of the rounding the result may be one step off, which the sum of both covers.
* 8-bit rows: a code is the nearest of value / scale, or the other neighbour where the fp32 error
  (relative, below 2^-16 in all cases) moves it over a border: half a step and that error.
"""
import math
import zlib

import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
TINY = {torch.bfloat16: 2.0**-133, torch.float16: 2.0**-24}  # the smallest step
U = 2.0**-24
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


def _gen(*key):
    return torch.Generator(device=DEV).manual_seed(zlib.crc32(repr(key).encode()))


def _rand(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _close(got, want, slack, dtype=torch.float32):
    """got (of `dtype`) is within one rounding of want, which itself may be off by `slack`."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    room = HALF.get(dtype, U) * (want.abs() + slack) + slack + TINY.get(dtype, 0.0)
    bad = ~((got - want).abs() <= room)
    assert not bool(bad.any()), (int(bad.sum()), got[bad][:3], want[bad][:3])


def _close8(rows8, want, slack):
    """Codes and scales of rows whose values `want` [rows, cols] may be off by `slack`, a share of
    their size."""
    top = want.abs().amax(-1)
    scale = (top / 448).clamp(min=2.0**-126)
    got = rows8.scales.double()
    assert bool(((got - scale).abs() <= (slack + 4 * U) * scale).all())
    v = want / got[..., None]  # what is rounded, from the scale that is stored
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0**-6)))
    step = torch.exp2(e - 3)
    off = (rows8.codes.double() - v.clamp(-448, 448)).abs()
    bad = off > step / 2 + (slack + 4 * U) * v.abs()
    assert not bool(bad.any()), (int(bad.sum()), rows8.codes[bad][:3].float(), v[bad][:3])


# ------------------------------------------------------------------------- rows in 8 bits
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 24), (5, 72), (17, 200), (9, 384), (33, 1032),
                                       (2, 8200), (1, 16384), (1000, 136)])
def test_quantize(rows, cols, dtype):
    g = _gen("q", rows, cols)
    x = _rand(g, rows, cols, dtype=dtype) * torch.exp(_rand(g, rows, 1, dtype=dtype))
    q = mrs.fp8_quantize(x)
    _close8(q, x.double(), 0.0)


def test_quantize_edges():
    x = torch.zeros(12, 64, device=DEV)
    x[1, 3] = 1e-45
    x[2, 3] = 3e38
    x[3, 0] = math.inf
    x[4, 1] = math.nan
    x[4, 2] = 5.0
    x[5] = -1.5
    x[6, :32] = -0.0
    x[7] = torch.linspace(-448, 448, 64)
    x[8, 5] = -math.inf
    x[9] = 2.0**-130
    q = mrs.fp8_quantize(x)
    bad = torch.tensor([3, 4, 8], device=DEV)
    assert torch.isnan(q.scales[bad]).all() and not q.codes[bad].view(torch.uint8).any()
    fine = torch.tensor([i for i in range(12) if i not in (3, 4, 8)], device=DEV)
    ok = mrs.Fp8Rows(q.codes.view(torch.uint8)[fine].view(F8), q.scales[fine])
    _close8(ok, x[fine].double(), 0.0)
    assert (q.scales[0] == 2.0**-126) and not q.codes[0].view(torch.uint8).any()


def test_quantize_views_and_three_dimensions():
    x = _rand(_gen("v"), 40, 512)
    for v in (x[:, :96], x[::3, 64:160], x[5:6, 8:40]):
        q, w = mrs.fp8_quantize(v), mrs.fp8_quantize(v.contiguous())
        assert torch.equal(q.codes.view(torch.uint8), w.codes.view(torch.uint8))
        assert torch.equal(q.scales, w.scales)
    three = torch.randn(4, 6, 64, device=DEV)
    q3 = mrs.fp8_quantize(three)
    assert q3.codes.shape == (4, 6, 64) and q3.scales.shape == (4, 6)
    _close8(q3, three.double(), 0.0)
    assert mrs.fp8_quantize(torch.empty(0, 64, device=DEV)).codes.shape == (0, 64)


# -------------------------------------------------------------------------------- the norm
def _ref_norm(x, residual, gain, parts, eps):
    T = x.shape[0] // parts
    total = x.double().view(T, parts, -1).sum(1)
    if residual is not None:
        total = total + residual.double()
    return total


SHAPES = [(1, 8, 1), (1, 3584, 16), (3, 24, 2), (7, 72, 3), (33, 256, 1), (5, 1000, 7),
          (130, 1024, 2), (2, 1032, 32), (9, 7168, 8), (2, 8200, 1), (1, 16384, 3), (600, 136, 5)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,cols,parts", SHAPES)
def test_norm(T, cols, parts, dtype):
    g = _gen("n", T, cols, parts)
    x = _rand(g, T * parts, cols, dtype=dtype)
    for with_res, gain_dtype in ((True, dtype), (False, torch.float32)):
        residual = _rand(g, T, cols, dtype=dtype, scale=2.0) if with_res else None
        gain = _rand(g, cols, dtype=gain_dtype) + 1
        out = mrs.rms_norm(x, gain, 1e-5, residual, parts, sum=True, fp8=True, rstd=True)
        total = _ref_norm(x, residual, gain, parts, 1e-5)
        size = x.double().abs().view(T, parts, -1).sum(1)
        if with_res:
            size = size + residual.double().abs()
        _close(out.sum, total, (parts + 1) * U * size, dtype)
        s = out.sum.double()  # the norm is that of what was stored
        rstd = 1 / torch.sqrt(s.square().mean(1) + 1e-5)
        _close(out.rstd, rstd, 40 * U * rstd)
        y = s * rstd[:, None] * gain.double()
        _close(out.y, y, 44 * U * y.abs(), dtype)
        _close8(out.rows8, y, 48 * U)
        # what is asked for changes nothing of the others
        only = mrs.rms_norm(x, gain, 1e-5, residual, parts)
        assert only.sum is None and only.rows8 is None and only.rstd is None
        assert torch.equal(only.y, out.y)


def test_norm_views_in_place_and_empty():
    g = _gen("p")
    wide, gain = _rand(g, 24, 1024), _rand(g, 512)
    x, residual = wide[::2, 256:768], wide[:6, 512:]
    got = mrs.rms_norm(x, gain, residual=residual, parts=2, sum=True)
    want = mrs.rms_norm(x.contiguous(), gain, residual=residual.contiguous(), parts=2, sum=True)
    assert torch.equal(got.y, want.y) and torch.equal(got.sum, want.sum)
    # the residual stream in place
    stream = residual.contiguous()
    y = torch.empty_like(stream)
    mrs.moe_rms_norm(x, gain, 1e-6, stream, 2, y, stream, None, None, None)
    assert torch.equal(stream, want.sum) and torch.equal(y, want.y)
    none = mrs.rms_norm(wide[:0], _rand(g, 1024), fp8=True)
    assert none.y.shape == (0, 1024)


def test_norm_of_zeros_infinities_and_large_rows():
    x = torch.zeros(5, 64, dtype=torch.bfloat16, device=DEV)
    x[1] = 1e15
    x[2, 3] = math.inf
    x[3, 4] = math.nan
    x[4] = -3.0
    gain = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    out = mrs.rms_norm(x, gain, 1e-6, fp8=True, rstd=True)
    assert not out.y[0].any() and out.rstd[0].item() == pytest.approx(1000.0, rel=1e-6)
    assert (out.y[1] == 1).all() and (out.y[4] == -1).all()
    assert torch.isnan(out.y[2, 3]) and torch.isnan(out.y[3]).all()
    assert torch.isnan(out.rows8.scales[2:4]).all()
    assert torch.isfinite(out.rows8.scales[[0, 1, 4]]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,cols,parts", SHAPES + [(3000, 64, 1), (2000, 2048, 1)])
def test_norm_backward(T, cols, parts, dtype):
    g = _gen("b", T, cols, parts)
    s, gain = _rand(g, T, cols, dtype=dtype), _rand(g, cols, dtype=dtype) + 1
    grad, rows = _rand(g, T, cols, dtype=dtype), _rand(g, T * parts, cols, dtype=dtype)
    more = _rand(g, T, cols, dtype=dtype)
    rstd = (s.float().square().mean(1) + 1e-5).rsqrt()
    for a, b, c in ((grad, rows, more), (grad, None, None), (None, rows, None)):
        out = mrs.rms_norm_backward(s, gain, rstd, a, b, parts, c)
        d, size = torch.zeros(2, T, cols, dtype=torch.float64, device=DEV)
        if a is not None:
            d, size = d + a.double(), size + a.double().abs()
        if b is not None:
            each = b.double().view(T, parts, cols)
            d, size = d + each.sum(1), size + each.abs().sum(1)
        r = rstd.double()[:, None]
        xh, dg = s.double() * r, d * gain.double()
        mean, sizes = (dg * xh).mean(1, keepdim=True), (size * gain.double() * xh).abs()
        dx = r * (dg - xh * mean)
        # d is off by parts u of its terms' sizes, the mean by its sum's levels too
        slack = r * ((parts + 6) * U * size * gain.double().abs() +
                     xh.abs() * (parts + 70) * U * sizes.mean(1, keepdim=True))
        if c is not None:
            dx = dx + c.double()
            slack = slack + 2 * U * c.double().abs()
        _close(out.x, dx, slack + 4 * U * dx.abs(), dtype)
        # a CTA's column sum: 32 tokens, then blocks of them, then CTAs: below 200 levels here
        _close(out.weight, (d * xh).sum(0), (parts + 200) * U * (size * xh.abs()).sum(0))
        none = mrs.rms_norm_backward(s, gain, rstd, a, b, parts, c, weight_grad=False)
        assert none.weight is None and torch.equal(none.x, out.x)


def test_norm_backward_is_the_gradient():
    g = _gen("d")
    T, cols, parts = 4, 64, 3
    x = torch.randn(T * parts, cols, generator=g, device=DEV, dtype=torch.float64)
    res = torch.randn(T, cols, generator=g, device=DEV, dtype=torch.float64)
    s = (x.view(T, parts, cols).sum(1) + res).bfloat16()
    gain = _rand(g, cols)
    grad = _rand(g, T, cols)
    rstd = (s.float().square().mean(1) + 1e-6).rsqrt()
    got = mrs.rms_norm_backward(s, gain, rstd, grad)

    def loss(v, w):
        return (v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w * grad.double()).sum()

    v, w = s.double(), gain.double()
    for i, j in ((0, 0), (1, 17), (3, 63)):
        h = torch.zeros_like(v)
        h[i, j] = 1e-4
        slope = (loss(v + h, w) - loss(v - h, w)) / 2e-4
        assert abs(got.x[i, j].item() - slope.item()) <= 2.0**-7 * (abs(slope.item()) + 0.05)
        h = torch.zeros_like(w)
        h[j] = 1e-4
        slope = (loss(v, w + h) - loss(v, w - h)) / 2e-4
        assert abs(got.weight[j].item() - slope.item()) <= 1e-5 * (abs(slope.item()) + 1)


def test_norm_backward_of_no_tokens():
    s = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    out = mrs.rms_norm_backward(s, torch.ones(64, dtype=torch.bfloat16, device=DEV),
                                torch.empty(0, device=DEV), s)
    assert not out.weight.any() and out.x.shape == (0, 64)


# -------------------------------------------------------------------- the gated activation
ROWS = [(1, 8), (16, 384), (5, 72), (33, 264), (3, 2048), (700, 136), (2, 8200), (1, 16384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", ROWS)
def test_swiglu(rows, cols, dtype):
    g = _gen("g", rows, cols)
    x = _rand(g, rows, 2 * cols, dtype=dtype, scale=3.0)
    x[0, :8] = torch.tensor([-90, -60, -20, 20, 60, 90, 0, -0.0], device=DEV).to(dtype)
    weights = torch.rand(rows, generator=g, device=DEV)
    a, b = x.double()[:, :cols], x.double()[:, cols:]
    for w in (weights, None):
        h = a * torch.sigmoid(a) * b
        if w is not None:
            h = h * w.double()[:, None]
        slack = (2.4 * a.abs() + 16) * U * h.abs() + 2.0**-126 * (a * b).abs()
        _close(mrs.swiglu(x, w), h, slack, dtype)
        _close8(mrs.swiglu(x, w, fp8=True), h, 240 * U)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", ROWS)
def test_swiglu_backward(rows, cols, dtype):
    g = _gen("h", rows, cols)
    x = _rand(g, rows, 2 * cols, dtype=dtype, scale=3.0)
    x[0, :8] = torch.tensor([-90, -60, -20, 20, 60, 90, 0, -0.0], device=DEV).to(dtype)
    grad = _rand(g, rows, cols, dtype=dtype)
    weights = torch.rand(rows, generator=g, device=DEV)
    a, b, d = x.double()[:, :cols], x.double()[:, cols:], grad.double()
    up, down = torch.sigmoid(a), torch.sigmoid(-a)
    for w in (weights, None):
        v = 1.0 if w is None else w.double()[:, None]
        got, gw = mrs.swiglu_backward(grad, x, w)
        ga, gb = v * d * b * up * (1 + a * down), v * d * a * up
        # 1 + a sig(-a) has terms up to 1 + |a sig(-a)|, which cancel near a = -1.28
        size = (v * d * b * up).abs() * (1 + (a * down).abs())
        small = 2.0**-126 * (1 + a.abs()) * (1 + b.abs()) * d.abs()
        _close(got[:, :cols], ga, (4.8 * a.abs() + 24) * U * size + small, dtype)
        _close(got[:, cols:], gb, (2.4 * a.abs() + 16) * U * gb.abs() + small, dtype)
        if w is None:
            assert gw is None
        else:
            terms = d * a * up * b
            _close(gw, terms.sum(1), ((2.4 * a.abs() + 80) * U * terms.abs() + small).sum(1))


def test_swiglu_backward_is_the_gradient():
    g = _gen("s")
    x, grad = _rand(g, 6, 32, dtype=torch.float16), _rand(g, 6, 16, dtype=torch.float16)
    w = torch.rand(6, generator=g, device=DEV)
    got, gw = mrs.swiglu_backward(grad, x, w)

    def loss(x, w):
        return (w[:, None] * torch.nn.functional.silu(x[:, :16]) * x[:, 16:] * grad.double()).sum()

    for i, j in ((0, 0), (2, 15), (5, 16), (3, 31)):
        h = torch.zeros(6, 32, dtype=torch.float64, device=DEV)
        h[i, j] = 1e-4
        slope = (loss(x.double() + h, w.double()) - loss(x.double() - h, w.double())) / 2e-4
        assert abs(got[i, j].item() - slope.item()) <= 2.0**-10 * (abs(slope.item()) + 0.01)
        h = torch.zeros(6, dtype=torch.float64, device=DEV)
        h[i] = 1e-4
        slope = (loss(x.double(), w.double() + h) - loss(x.double(), w.double() - h)) / 2e-4
        assert abs(gw[i].item() - slope.item()) <= 1e-5 * (abs(slope.item()) + 1)


def test_swiglu_views_and_buffers():
    g = _gen("w")
    wide = _rand(g, 20, 512)
    x = wide[::2, 128:384]
    assert torch.equal(mrs.swiglu(x), mrs.swiglu(x.contiguous()))
    out = torch.full((12, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    got = mrs.swiglu(x, out=out[:10])
    assert got.data_ptr() == out.data_ptr() and (out[10:] == 7).all()
    q, y = mrs.Fp8Rows.allocate(10, 128, device=DEV), torch.empty(10, 128, dtype=x.dtype, device=DEV)
    mrs.moe_swiglu(x, None, y, q.codes, q.scales)
    assert torch.equal(y, out[:10])
    grad = _rand(g, 10, 128)
    a, _ = mrs.swiglu_backward(grad, x)
    b, _ = mrs.swiglu_backward(grad, x.contiguous())
    assert torch.equal(a, b)
    assert mrs.swiglu(wide[:0]).shape == (0, 256)


# ----------------------------------------------------------------------- calls and refusals
def test_rows_past_32_bit_offsets():
    rows, cols = 140000, 16384  # more than 2^31 elements
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-3:] = torch.randn(3, cols, device=DEV)
    last = x[-3:].clone()
    gain = torch.ones(cols, dtype=torch.bfloat16, device=DEV)
    out = mrs.rms_norm(x, gain, fp8=True)
    one = mrs.rms_norm(last, gain, fp8=True)
    assert torch.equal(out.y[-3:], one.y)
    assert torch.equal(out.rows8.codes[-3:].view(torch.uint8), one.rows8.codes.view(torch.uint8))
    assert torch.equal(mrs.swiglu(x)[-3:], mrs.swiglu(last))
    del out
    rstd = torch.ones(rows, device=DEV)
    got = mrs.rms_norm_backward(x, gain, rstd, x, weight_grad=False)
    want = mrs.rms_norm_backward(last, gain, rstd[:3], last, weight_grad=False)
    assert torch.equal(got.x[-3:], want.x)


def test_on_another_stream_and_in_a_graph():
    g = _gen("c")
    x, gain = _rand(g, 64, 1024), _rand(g, 1024)
    want = mrs.rms_norm(x, gain, fp8=True, sum=True, rstd=True)
    wh = mrs.swiglu(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mrs.rms_norm(x, gain, fp8=True, sum=True, rstd=True, stream=side)
    gh = mrs.swiglu(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in ((got.y, want.y), (got.sum, want.sum), (got.rstd, want.rstd), (gh, wh)):
        assert torch.equal(a, b)
    grads = mrs.rms_norm_backward(want.sum, gain, want.rstd, x)
    out = mrs.NormGrads.allocate(64, 1024, device=DEV)
    buf = mrs.NormBuffers.allocate(64, 1024, fp8=True, sum=True, rstd=True, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mrs.rms_norm(x, gain, out=buf)
        mrs.rms_norm_backward(buf.sum, gain, buf.rstd, x, out=out)
    for _ in range(3):
        for t in (*buf.tensors, out.x, out.weight):
            t.view(torch.uint8).fill_(255)
        graph.replay()
        assert torch.equal(buf.y, want.y) and torch.equal(out.x, grads.x)
        assert torch.equal(out.weight, grads.weight)


def test_refusals_on_the_device():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="multiple of 3 parts"):
        mrs.rms_norm(x, w, parts=3)
    with pytest.raises(ValueError, match="weight must be"):
        mrs.rms_norm(x, w.half())
    with pytest.raises(ValueError, match="weight holds"):
        mrs.rms_norm(x, w[:32].contiguous())
    with pytest.raises(ValueError, match="residual must be"):
        mrs.rms_norm(x, w, residual=x[:2])
    with pytest.raises(ValueError, match="x must be bfloat16"):
        mrs.rms_norm(x.float(), w)
    with pytest.raises(ValueError, match="dense rows"):
        mrs.rms_norm(x.t(), w[:4].contiguous())
    with pytest.raises(ValueError, match="out is for"):
        mrs.rms_norm(x, w, out=mrs.NormBuffers.allocate(5, 64, device=DEV))
    with pytest.raises(ValueError, match="grad must be"):
        mrs.rms_norm_backward(x, w, torch.ones(4, device=DEV), x[:2])
    with pytest.raises(mrs.RouteSortError):
        mrs.rms_norm_backward(x, w, torch.ones(4, device=DEV))
    with pytest.raises(ValueError, match="weights holds"):
        mrs.swiglu(x, torch.ones(3, device=DEV))
    with pytest.raises(ValueError, match="out must be"):
        mrs.swiglu(x, out=x)
    with pytest.raises(ValueError, match="scales must be"):
        mrs.Fp8Rows(torch.empty(4, 64, dtype=F8, device=DEV), torch.empty(3, device=DEV))
    with pytest.raises(mrs.RouteSortError):
        mrs.fp8_quantize(torch.zeros(4, 12, device=DEV))
