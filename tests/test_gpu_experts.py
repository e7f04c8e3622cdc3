"""MXFP4 rows and the experts' products on a GB300, against plain float64 implementations.

Quantisation is exact arithmetic (a power-of-two scaling and one rounding to a grid), so codes and
scale bytes are compared bit for bit with a search over the grid.  A product of two codes and two
scales is exact in fp32 (4 significant bits); a sum of cols of them in fp32 is within
cols * 2^-24 * sum |x w| of the float64 sum in any order, and a matrix unit that keeps at least 24
bits of every aligned term stays within cols * 2^-23 * sum |x w|, the tolerance used.  The weight
adds 2^-24 of the value, a bf16 output half a step, 2^-8 of the value.
"""
import math

import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


def _ref_quantise(x):
    """(codes of each element, scale byte of each block) by search, in float64 on the CPU."""
    b = x.detach().cpu().double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    m, e = torch.frexp(torch.where(bad | (top == 0), 1.0, top))
    e = torch.where(top == 0, -127, (e - 3).clamp(-127, 125)).long()
    v = (b.abs() * torch.pow(2.0, -e.double())[..., None]).nan_to_num(0.0, 0.0, 0.0)
    d = (v[..., None] - GRID).abs()
    near = d == d.amin(-1, keepdim=True)
    even = torch.arange(8) % 2 == 0
    code = torch.where((near & even).any(-1), (near & even).int().argmax(-1), near.int().argmax(-1))
    code = code + 8 * torch.signbit(b).long()
    code = torch.where(bad[..., None], 0, code)
    return code.flatten(-2), torch.where(bad, 255, e + 127)


def _unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()


def _value(codes, scales, cols):
    c = _unpack(codes.cpu())
    s = scales.cpu()[..., : cols // 32].double()
    v = GRID[c & 7] * torch.where(c >= 8, -1.0, 1.0)
    step = torch.where(s == 255, math.nan, torch.pow(2.0, s - 127))
    return (v.unflatten(-1, (-1, 32)) * step[..., None]).flatten(-2)


def _check_quantise(x):
    q = mrs.mxfp4_quantize(x)
    torch.cuda.synchronize()
    code, byte = _ref_quantise(x)
    cols = x.shape[-1]
    assert torch.equal(_unpack(q.codes.cpu()), code)
    assert torch.equal(q.scales.cpu()[..., : cols // 32].long(), byte)
    assert not q.scales[..., cols // 32:].any()
    for dtype in (torch.bfloat16, torch.float32):
        y = mrs.mxfp4_dequantize(q, dtype=dtype).cpu().double()
        ref = _value(q.codes, q.scales, cols)
        assert torch.equal(torch.isnan(y), torch.isnan(ref))
        assert torch.equal(y.nan_to_num(), ref.nan_to_num())
    return q


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (5, 96), (7, 128), (1, 3584), (257, 416),
                                       (1000, 160), (2, 32768)])
def test_quantise(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    x = x.clamp(-60000, 60000)
    _check_quantise(x.to(dtype).to(DEV))


def test_quantise_every_bf16():
    # each bf16 pattern beside a block maximum that makes it land on and between the codes
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = torch.where(torch.isfinite(bits), bits, 0.0)
    x = torch.zeros(65536, 32, dtype=torch.bfloat16)
    x[:, 5] = bits
    for k, f in [(0, 1.0), (1, 2.5), (9, -0.625), (31, 1.75)]:
        x[:, k] = (bits.float() * f).clamp(-3e38, 3e38).bfloat16()
    _check_quantise(x.to(DEV))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantise_edges(dtype):
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x = torch.zeros(16, 64, dtype=dtype)
    x[0, 0] = big
    x[1, 3] = tiny
    x[2, 3] = tiny / 64  # subnormal
    x[3, 40] = math.inf
    x[4, 1] = math.nan
    x[5, :32] = -0.0
    x[6] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 8).to(dtype)
    x[7] = -x[6]
    x[8, 0] = -math.inf
    x[8, 1] = 1.0
    x[9] = 7.984375
    _check_quantise(x.to(DEV))


def test_quantise_strided_rows_and_views():
    x = torch.randn(40, 512, device=DEV).bfloat16()
    for v in (x[:, :96], x[::3, 64:160], x[5:6, 8:40]):
        q = mrs.mxfp4_quantize(v)
        w = mrs.mxfp4_quantize(v.contiguous())
        assert torch.equal(q.codes, w.codes) and torch.equal(q.scales, w.scales)
    y = torch.full((40, 512), 7.0, device=DEV)
    q = mrs.mxfp4_quantize(x[:, :96])
    mrs.mxfp4_dequantize(q, out=y[:, 16:112])
    assert torch.equal(y[:, 16:112].double().cpu(), _value(q.codes, q.scales, 96))
    assert (y[:, :16] == 7).all() and (y[:, 112:] == 7).all()
    three = torch.randn(4, 6, 64, device=DEV)
    q3 = mrs.mxfp4_quantize(three)
    assert q3.codes.shape == (4, 6, 32) and mrs.mxfp4_dequantize(q3).shape == (4, 6, 64)


def test_rows_past_32_bit_offsets():
    # more than 2^31 elements: the last rows, against the same rows quantised alone
    rows, cols = 70000, 32768
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-3:] = torch.randn(3, cols, device=DEV)
    q = mrs.Mxfp4Rows.allocate(rows, cols, device=DEV)
    mrs.mxfp4_quantize(x, out=q)
    one = mrs.mxfp4_quantize(x[-3:].clone())
    assert torch.equal(q.codes[-3:], one.codes) and torch.equal(q.scales[-3:], one.scales)


# ------------------------------------------------------------------------------ products
def _rows(g, rows, cols, spread=1.0):
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g))
    return mrs.mxfp4_quantize(x.to(DEV))


def _routes(g, T, E, K, dist):
    if dist == "uniform":
        return torch.rand(T, E, generator=g).topk(K, dim=1).indices.int()
    if dist == "one":
        return torch.full((T, K), E - 1, dtype=torch.int32)
    ids = torch.randint(0, E, (T, K), generator=g).int()  # repeats inside a token, drops
    ids.view(-1)[:: 4] = -1
    return ids


def _sorted(ids, w, E, B):
    T, K = ids.shape
    out = mrs.RouteSortBuffers.allocate(T, E, K, B, device=DEV)
    mrs.moe_sort(ids.to(DEV), w.to(DEV), E, B, out.sorted_token_ids, out.sorted_weights,
                 out.expert_ids, out.num_tokens_post_pad, out.workspace)
    return out


def _ref_product(ids, w, x, W, cols, per_route):
    T, K = ids.shape
    xv, wv = _value(x.codes, x.scales, cols).to(DEV), _value(W.codes, W.scales, cols).to(DEV)
    N = wv.shape[1]
    y = torch.zeros(T * K, N, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(y)
    flat = ids.reshape(-1).to(DEV)
    for e in flat.unique().tolist():
        if e < 0:
            continue
        r = (flat == e).nonzero()[:, 0]
        a = xv[r if per_route else r // K]
        y[r] = a @ wv[e].T
        mag[r] = a.abs() @ wv[e].abs().T
    if w is not None:
        s = w.reshape(-1, 1).double().to(DEV)
        y, mag = y * s, mag * s.abs()
    return y, mag


def _check_product(T, E, K, cols, N, B, dist="uniform", per_route=False, weighted=True,
                   dtype=torch.float32, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed + T + E + cols + N + B)
    ids = _routes(g, T, E, K, dist)
    w = torch.randn(T, K, generator=g)
    x = _rows(g, T * K if per_route else T, cols, spread)
    W = _rows(g, E * N, cols, spread)
    W = mrs.Mxfp4Rows(W.codes.view(E, N, -1), W.scales.view(E, N, -1))
    m = _sorted(ids, w, E, B)
    out = torch.full((T * K, N), 12345.0, dtype=dtype, device=DEV)
    ws = torch.zeros(mrs.moe_experts_mxfp4_workspace_bytes(T, E, K, B), dtype=torch.uint8,
                     device=DEV)
    mrs.experts_mxfp4(x, W, T, K, B, m.sorted_token_ids, m.expert_ids, m.num_tokens_post_pad,
                      m.sorted_weights if weighted else None, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0
    y, mag = _ref_product(ids, w if weighted else None, x, W, cols, per_route)
    dropped = (ids.reshape(-1) < 0).to(DEV)
    assert (out[dropped] == 12345.0).all()
    err = (out.double() - y).abs()[~dropped]
    tol = cols * 2.0 ** -23 * mag + 2.0 ** -24 * y.abs() + 1e-38
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (y.abs() + tol)
    bad = err > tol[~dropped]
    assert not bad.any(), (int(bad.sum()), float(err.max()))
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [1, 2, 8, 16, 32, 64, 128, 256, 1024])
def test_product_block_sizes(B, dtype):
    _check_product(37, 6, 3, 256, 136, B, dtype=dtype)


@pytest.mark.parametrize("cols", [32, 64, 96, 128, 160, 256, 288, 384, 512, 544, 1120, 3584])
@pytest.mark.parametrize("B", [16, 128])
def test_product_row_lengths(cols, B):
    _check_product(21, 5, 2, cols, 128, B)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [8, 16, 128, 256, 1024])
@pytest.mark.parametrize("T,dist", [(1500, "uniform"), (7000, "uniform"), (9000, "uniform"),
                                    (9000, "one"), (3000, "drops"), (9100, "drops")])
def test_product_of_long_rows_and_many_tokens(T, dist, B, dtype):
    # tiles of 256 outputs fill tensor memory: one ends before the next one starts, several times per
    # CTA, in windows, in single blocks and in parts of blocks
    _check_product(T, 4, 2, 2080, 1000, B, dist, dtype=dtype)
    _check_product(T, 4, 2, 1056, 520, B, dist, dtype=dtype)


@pytest.mark.parametrize("N", [8, 16, 72, 120, 128, 136, 256, 264, 768])
def test_product_output_widths(N):
    _check_product(19, 4, 2, 192, N, 16)
    _check_product(150, 4, 2, 192, N, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("T,E,K,cols,N,B", [
    (1, 896, 16, 3584, 768, 16), (1, 1, 1, 32, 8, 1), (2, 64, 6, 512, 256, 32),
    (129, 3, 1, 384, 200, 128), (700, 16, 4, 384, 1024, 128), (300, 2, 2, 1024, 384, 256),
    (64, 4096, 8, 64, 16, 16),
])
@pytest.mark.parametrize("per_route", [False, True])
def test_product_shapes(T, E, K, cols, N, B, per_route):
    _check_product(T, E, K, cols, N, B, per_route=per_route, dtype=torch.bfloat16)


@pytest.mark.parametrize("T,E,K,cols,N,B", [
    (2000, 8, 4, 640, 1536, 64),    # wide tiles, one a unit
    (8000, 8, 4, 320, 1536, 64),    # wide tiles, several a unit, the last unit of a block shorter
    (8000, 8, 4, 512, 1432, 64),    # the same with a ragged last tile
    (20000, 8, 4, 96, 256, 64),     # narrow tiles, several a unit
    (9000, 8, 4, 768, 768, 128),    # the most steps whose rows could stay for narrow tiles
    (3000, 700, 8, 256, 640, 16),   # many experts of few rows
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_many_tiles(T, E, K, cols, N, B, dtype):
    _check_product(T, E, K, cols, N, B, dtype=dtype, per_route=dtype == torch.float32)


@pytest.mark.parametrize("B", [1, 2, 4, 16, 32, 64])
@pytest.mark.parametrize("T,E,K", [(70, 2, 1), (300, 3, 2), (1000, 40, 4)])
def test_product_blocks_that_share_a_tile(T, E, K, B):
    # runs of one expert's blocks that start, end and are cut inside windows of 128 rows
    _check_product(T, E, K, 288, 200, B, dist="drops" if K == 4 else "uniform")


@pytest.mark.parametrize("dist", ["one", "drops"])
@pytest.mark.parametrize("B", [16, 64, 128])
@pytest.mark.parametrize("weighted", [False, True])
def test_product_routes(dist, B, weighted):
    _check_product(200, 9, 4, 320, 160, B, dist=dist, weighted=weighted, per_route=weighted)


def test_product_scales_of_any_size():
    _check_product(50, 4, 2, 256, 128, 32, spread=9.0)


def test_all_routes_dropped_and_no_tokens():
    T, E, K, cols, N, B = 5, 4, 2, 64, 16, 16
    g = torch.Generator().manual_seed(0)
    W = _rows(g, E * N, cols)
    W = mrs.Mxfp4Rows(W.codes.view(E, N, -1), W.scales.view(E, N, -1))
    m = _sorted(torch.full((T, K), -1, dtype=torch.int32), torch.ones(T, K), E, B)
    out = mrs.experts_mxfp4(_rows(g, T, cols), W, T, K, B, m.sorted_token_ids, m.expert_ids,
                            m.num_tokens_post_pad)
    assert not out.any()
    empty = mrs.Mxfp4Rows.allocate(0, cols, device=DEV)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert mrs.experts_mxfp4(empty, W, 0, K, B, z, z, z).shape == (0, N)


def test_nan_scale_reaches_its_rows_only():
    T, E, K, cols, N, B = 40, 4, 2, 256, 128, 32
    g = torch.Generator().manual_seed(3)
    ids = _routes(g, T, E, K, "uniform")
    x = _rows(g, T, cols)
    x.scales[7, 3] = 255
    W = _rows(g, E * N, cols)
    W = mrs.Mxfp4Rows(W.codes.view(E, N, -1), W.scales.view(E, N, -1))
    W.scales[2, 5, 0] = 255
    m = _sorted(ids, torch.ones(T, K), E, B)
    out = mrs.experts_mxfp4(x, W, T, K, B, m.sorted_token_ids, m.expert_ids,
                            m.num_tokens_post_pad, dtype=torch.float32)
    nan = torch.zeros(T * K, N, dtype=torch.bool)
    nan[7 * K: 8 * K] = True
    nan[(ids.reshape(-1) == 2), 5] = True
    assert torch.equal(torch.isnan(out).cpu(), nan)


def test_padding_scale_bytes_are_not_used():
    T, E, K, N, B = 20, 4, 2, 64, 16
    g = torch.Generator().manual_seed(6)
    for cols in (32, 96, 160, 288):
        ids = _routes(g, T, E, K, "uniform")
        x, W = _rows(g, T, cols), _rows(g, E * N, cols)
        W = mrs.Mxfp4Rows(W.codes.view(E, N, -1), W.scales.view(E, N, -1))
        m = _sorted(ids, torch.ones(T, K), E, B)
        lists = (m.sorted_token_ids, m.expert_ids, m.num_tokens_post_pad)
        a = mrs.experts_mxfp4(x, W, T, K, B, *lists, dtype=torch.float32)
        x.scales[:, cols // 32:] = 255
        W.scales[:, :, cols // 32:] = 255
        assert torch.equal(a, mrs.experts_mxfp4(x, W, T, K, B, *lists, dtype=torch.float32))


def test_bad_expert_ids_and_list_entries_are_skipped():
    T, E, K, cols, N, B = 32, 4, 1, 128, 64, 16
    g = torch.Generator().manual_seed(4)
    ids = (torch.arange(T)[:, None] % E).int()
    x, W = _rows(g, T, cols), _rows(g, E * N, cols)
    W = mrs.Mxfp4Rows(W.codes.view(E, N, -1), W.scales.view(E, N, -1))
    m = _sorted(ids, torch.ones(T, K), E, B)
    good = mrs.experts_mxfp4(x, W, T, K, B, m.sorted_token_ids, m.expert_ids,
                             m.num_tokens_post_pad)
    for bad_id in (-3, E, 1 << 30):
        eid, sid = m.expert_ids.clone(), m.sorted_token_ids.clone()
        eid[1] = bad_id                # expert 1's block
        sid[0], sid[1] = -5, 1 << 30   # two rows of expert 0
        out = torch.full((T, N), 9.0, dtype=torch.bfloat16, device=DEV)
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        mrs.experts_mxfp4(x, W, T, K, B, sid, eid, m.num_tokens_post_pad, out=out, workspace=ws)
        lost = torch.zeros(T, dtype=torch.bool)
        lost[1::E] = True
        lost[0] = lost[4] = True
        assert (out[lost.to(DEV)] == 9.0).all()
        assert torch.equal(out[~lost.to(DEV)], good[~lost.to(DEV)])
        assert int(ws[:4].view(torch.int32)) == mrs.DEVICE_BAD_EXPERT_ID
    for npp in (-1, 0, 1 << 30):  # a length outside the list is cut to it
        out = torch.full((T, N), 9.0, dtype=torch.bfloat16, device=DEV)
        n = torch.tensor([npp], dtype=torch.int32, device=DEV)
        sid = torch.full_like(m.sorted_token_ids, T)
        mrs.experts_mxfp4(x, W, T, K, B, sid, torch.zeros_like(m.expert_ids), n, out=out)
        assert (out == 9.0).all()


def test_same_bits_every_call_graph_and_stream():
    T, E, K, cols, N, B = 300, 16, 4, 512, 384, 32
    g = torch.Generator().manual_seed(5)
    ids = _routes(g, T, E, K, "uniform")
    x, W = _rows(g, T, cols), _rows(g, E * N, cols)
    W = mrs.Mxfp4Rows(W.codes.view(E, N, -1), W.scales.view(E, N, -1))
    m = _sorted(ids, torch.rand(T, K), E, B)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    outs = [torch.empty(T * K, N, dtype=torch.bfloat16, device=DEV) for _ in range(3)]

    def call(out):
        mrs.experts_mxfp4(x, W, T, K, B, m.sorted_token_ids, m.expert_ids, m.num_tokens_post_pad,
                          m.sorted_weights, out=out, workspace=ws)

    call(outs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[1])
    graph.replay()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # at the same time, on the same workspace
        call(outs[2])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("T", [1, 40, 300])
def test_a_moe_layer_from_router_to_output(T):
    """Route, quantise, first product, activation, quantise, second product, sum over experts:
    the 4-bit operator this library's metadata feeds, at reduced sizes, against float64 on the
    same quantised values."""
    E, G, Kg, K, H, I, B, R = 64, 8, 4, 6, 256, 96, 16, 2.5
    g = torch.Generator().manual_seed(T)
    logits = torch.randn(T, E, generator=g).bfloat16().to(DEV)
    bias = (0.1 * torch.rand(E, generator=g)).to(DEV)
    hidden = torch.randn(T, H, generator=g).bfloat16().to(DEV)
    W1 = mrs.mxfp4_quantize((torch.randn(E, 2 * I, H, generator=g) / H ** 0.5).bfloat16().to(DEV))
    W2 = mrs.mxfp4_quantize((torch.randn(E, H, I, generator=g) / I ** 0.5).bfloat16().to(DEV))
    r = mrs.route_sort(logits, bias, G, Kg, K, R, B)
    x = mrs.mxfp4_quantize(hidden)
    lists = (r.sorted_token_ids, r.expert_ids, r.num_tokens_post_pad)
    h = mrs.experts_mxfp4(x, W1, T, K, B, *lists, dtype=torch.float32)
    act = (torch.nn.functional.silu(h[:, :I]) * h[:, I:]).bfloat16()
    a = mrs.mxfp4_quantize(act)
    y = mrs.experts_mxfp4(a, W2, T, K, B, *lists, sorted_weights=r.sorted_weights,
                          dtype=torch.float32).view(T, K, H).sum(1)
    ids, w = r.topk_ids.cpu(), r.topk_weights.cpu()
    h64, mag = _ref_product(ids, None, x, W1, H, False)
    assert ((h.double() - h64).abs() <= H * 2.0 ** -23 * mag + 1e-38).all()
    y64, mag = _ref_product(ids, w, a, W2, I, True)
    y64, mag = y64.view(T, K, H).sum(1), mag.view(T, K, H).sum(1)
    assert ((y.double() - y64).abs() <= (I * 2.0 ** -23 + K * 2.0 ** -23) * mag + 1e-38).all()


@pytest.mark.parametrize("B,cols", [(16, 512), (128, 2048)])
def test_waits_that_give_up_are_reported_and_leave_the_next_call_right(B, cols):
    T, E, K, N = 60, 4, 2, 256
    g = torch.Generator().manual_seed(7)
    ids = _routes(g, T, E, K, "uniform")
    x, W = _rows(g, T, cols), _rows(g, E * N, cols)
    W = mrs.Mxfp4Rows(W.codes.view(E, N, -1), W.scales.view(E, N, -1))
    m = _sorted(ids, torch.ones(T, K), E, B)
    lists = (m.sorted_token_ids, m.expert_ids, m.num_tokens_post_pad)
    good = mrs.experts_mxfp4(x, W, T, K, B, *lists)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    try:
        mrs.moe_route_sort_debug_set(mrs.DEBUG_WAIT_LIMIT_NS, 0)
        out = torch.full_like(good, 3.0)
        mrs.experts_mxfp4(x, W, T, K, B, *lists, out=out, workspace=ws)
        torch.cuda.synchronize()
    finally:
        mrs.moe_route_sort_debug_set(mrs.DEBUG_WAIT_LIMIT_NS, -1)
    assert int(ws[:4].view(torch.int32)) == 2  # MOE_RS_DEVICE_WAIT_TIMEOUT
    ws.zero_()
    again = mrs.experts_mxfp4(x, W, T, K, B, *lists, workspace=ws)
    assert torch.equal(again, good) and int(ws[:4].view(torch.int32)) == 0


def test_a_call_on_another_stream_makes_its_buffers_there():
    # the current stream is busy for a while; what the calls allocate must not wait for it, nor be
    # cleared or filled after the kernels on the other stream have run
    T, E, K, cols, N, B = 50, 8, 2, 128, 64, 16
    g = torch.Generator().manual_seed(8)
    ids = _routes(g, T, E, K, "uniform")
    x, W = _rows(g, T, cols), _rows(g, E * N, cols)
    W = mrs.Mxfp4Rows(W.codes.view(E, N, -1), W.scales.view(E, N, -1))
    m = _sorted(ids, torch.ones(T, K), E, B)
    lists = (m.sorted_token_ids, m.expert_ids, m.num_tokens_post_pad)
    want = mrs.experts_mxfp4(x, W, T, K, B, *lists)
    three = torch.randn(4, 64, 6, generator=g).to(DEV).transpose(1, 2)  # copied to become rows
    want3 = mrs.mxfp4_quantize(three.contiguous())
    back3 = mrs.mxfp4_dequantize(want3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        torch.cuda._sleep(50_000_000)
        got = mrs.experts_mxfp4(x, W, T, K, B, *lists, stream=stream)
        got3 = mrs.mxfp4_quantize(three, stream=stream)
        got_back = mrs.mxfp4_dequantize(got3, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert torch.equal(got3.codes, want3.codes) and torch.equal(got3.scales, want3.scales)
        assert torch.equal(got_back, back3)


def test_rows_whose_memory_was_exchanged():
    # a caller may offload and bring back the memory behind a tensor that a container holds
    x = torch.randn(64, 512, device=DEV)
    q = mrs.mxfp4_quantize(x)
    want = mrs.mxfp4_dequantize(q)
    host = q.codes.cpu()
    size = q.codes.untyped_storage().nbytes()
    q.codes.untyped_storage().resize_(0)
    with pytest.raises(mrs.RouteSortError):
        mrs.mxfp4_dequantize(q)
    keep = torch.full((size,), 255, dtype=torch.uint8, device=DEV)  # what was there is other data
    q.codes.untyped_storage().resize_(size)
    q.codes.copy_(host)
    assert torch.equal(mrs.mxfp4_dequantize(q), want)
    assert (keep == 255).all()
