"""Calls of the training and experts operators that their documentation allows beside the common
ones, on a GB300."""
import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


def _router(T, E, K, seed=0):
    g = torch.Generator().manual_seed(seed)
    logits = (1.5 * torch.randn(T, E, generator=g)).bfloat16()
    ids = torch.rand(T, E, generator=g).topk(K, dim=1).indices.int()
    return logits.to(DEV), ids.to(DEV)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,K", [(64, 6), (129, 5), (2056, 8)])
def test_the_loss_gradient_does_not_need_the_ids(E, K, softmax):
    # the same call with and without ids: the routes only steer the weights' term
    logits, ids = _router(200, E, K)
    counts = mrs.balance_loss(logits, ids, 0.5, softmax=softmax).counts
    term = dict(softmax=softmax, grad_loss=torch.ones(1, device=DEV), counts=counts, coef=0.5,
                dtype=torch.float32)
    want = mrs.route_backward(logits, ids, **term)
    assert torch.equal(mrs.route_backward(logits, None, topk=K, **term), want)
    assert want.any()


def _layer(T, E, K, cols, N, B, seed=0):
    """Rows, weights and the lists of a small layer, every token to different experts."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).topk(K, dim=1).indices.int().to(DEV)
    x = mrs.mxfp4_quantize(torch.randn(T, cols, generator=g).to(DEV))
    w = mrs.mxfp4_quantize(torch.randn(E, N, cols, generator=g).to(DEV))
    m = mrs.RouteSortBuffers.allocate(T, E, K, B, device=DEV)
    mrs.moe_sort(ids, torch.ones(T, K, device=DEV), E, B, m.sorted_token_ids, m.sorted_weights,
                 m.expert_ids, m.num_tokens_post_pad, m.workspace)
    return x, w, (m.sorted_token_ids, m.expert_ids, m.num_tokens_post_pad)


def test_device_errors_show_on_every_path_of_the_products():
    T, E, K, cols, N, B = 32, 4, 2, 128, 64, 16
    x, w, (sid, eid, npp) = _layer(T, E, K, cols, N, B)
    bad = eid.clone()
    bad[1] = E + 7
    own = mrs.ExpertsWorkspace.allocate(T, E, K, B, device=DEV)
    mrs.experts_status(DEV, clear=True)
    good = mrs.experts_mxfp4(x, w, T, K, B, sid, eid, npp)
    assert torch.equal(mrs.experts_mxfp4(x, w, T, K, B, sid, eid, npp, workspace=own), good)
    assert mrs.experts_status(DEV) == 0 and own.status_word() == 0
    # with a workspace the bits are that one's alone
    mrs.experts_mxfp4(x, w, T, K, B, sid, bad, npp, workspace=own)
    assert own.status_word() == mrs.DEVICE_BAD_EXPERT_ID and mrs.experts_status(DEV) == 0
    own.clear()
    assert own.status_word() == 0
    # without one, of the device: kept over good calls, cleared when asked; any stream, a graph too
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mrs.experts_mxfp4(x, w, T, K, B, sid, bad, npp, stream=side)
    mrs.experts_mxfp4(x, w, T, K, B, sid, eid, npp)
    assert mrs.experts_status(DEV) == mrs.DEVICE_BAD_EXPERT_ID
    assert mrs.experts_status(DEV, clear=True) == mrs.DEVICE_BAD_EXPERT_ID
    assert mrs.experts_status(DEV) == 0 and own.status_word() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mrs.experts_mxfp4(x, w, T, K, B, sid, bad, npp)
    assert mrs.experts_status(DEV) == 0
    graph.replay()
    assert mrs.experts_status(DEV, clear=True) == mrs.DEVICE_BAD_EXPERT_ID
    assert not torch.equal(got, good)
    try:
        mrs.moe_route_sort_debug_set(mrs.DEBUG_WAIT_LIMIT_NS, 0)
        mrs.experts_mxfp4(x, w, T, K, B, sid, eid, npp)
        torch.cuda.synchronize()
    finally:
        mrs.moe_route_sort_debug_set(mrs.DEBUG_WAIT_LIMIT_NS, -1)
    assert mrs.experts_status(DEV, clear=True) == mrs.DEVICE_WAIT_TIMEOUT
    assert torch.equal(mrs.experts_mxfp4(x, w, T, K, B, sid, eid, npp), good)
    assert mrs.experts_status(DEV) == 0


def _gpu_time(call, n=10):
    for _ in range(3):
        call()
    start, end = torch.cuda.Event(True), torch.cuda.Event(True)
    start.record()
    for _ in range(n):
        call()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / n  # ms


@pytest.mark.parametrize("where", ["behind padding", "in the middle", "at the start", "at the end",
                                   "two clumps"])
@pytest.mark.parametrize("softmax", [False, True])
def test_any_number_of_empty_sequences(where, softmax):
    # 60000 empty sequences change the mean over sequences and nothing else, and are stepped over
    # by searching: one after another they took up to 12 ms at 8192 tokens
    T, E, K, n = 3000, 64, 6, 60000
    logits, ids = _router(T, E, K)
    a, b = T // 3, T - 10
    few = {"behind padding": [b, T], "in the middle": [0, a, T], "at the start": [0, a, T],
           "at the end": [0, a, b], "two clumps": [5, a, b]}[where]
    many = {"behind padding": [b] * n + [T], "in the middle": [0] + [a] * n + [T],
            "at the start": [0] * n + [a, T], "at the end": [0, a] + [b] * n,
            "two clumps": [5] + [a] * n + [b] * (n // 16)}[where]
    got, one = [], torch.ones(1, device=DEV)
    for offsets in (few, many):
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        S = len(offsets) - 1
        out = mrs.BalanceBuffers.allocate(T, E, S, device=DEV)
        grad = torch.empty(T, E, device=DEV)

        def loss():
            # (coef times S: a sequence weighs the same in both)
            mrs.balance_loss(logits, ids, 0.5 * S, softmax=softmax, seq_offsets=off, out=out)

        def backward():
            mrs.route_backward(logits, ids, None, 1.0, softmax, one, out.counts, 0.5 * S, off,
                               out=grad)

        times = [_gpu_time(loss), _gpu_time(backward)]
        full = [i for i in range(S) if offsets[i + 1] > offsets[i]]
        got.append((out.loss.item(), out.counts[full], out.mean_probs[full], grad, times))
        assert int(out.counts.sum()) == int(out.counts[full].sum())
        assert not out.mean_probs.sum(1)[[i for i in (0, S // 2, S - 1) if i not in full]].any()
    (l0, c0, m0, g0, t0), (l1, c1, m1, g1, t1) = got
    assert torch.equal(c0, c1) and torch.equal(m0, m1)
    # one more rounding of coef / S, and sums of the same terms in another order
    assert abs(l0 - l1) <= 2.0 ** -20 * abs(l0)
    assert torch.all((g0 - g1).abs() <= 2.0 ** -20 * g0.abs() + 1e-30)
    # 60000 rows of counts and means are written (9 times the short call's 11 us); the gradient
    # only searches (the same 8 us)
    assert t1[0] <= 30 * t0[0] and t1[1] <= 10 * t0[1], (t0, t1)


@pytest.mark.parametrize("softmax", [False, True])
def test_the_means_of_many_tokens(softmax):
    # equal logits: every probability is 1 / 56, a sum's roundings all go the same way, and one
    # addition per token (6900 a group of warps) was off by 7.7e-5.  Now: a probability within
    # 2^-22, sums 128 + 54 additions deep, 16 groups, 19 + 8 CTAs, each 2^-24: 2^-16 in all; the loss
    # adds 56 terms to that.
    T, E, K = 1 << 24, 56, 2
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    ids = torch.randint(0, E, (T, K), dtype=torch.int32, device=DEV)
    out = mrs.balance_loss(logits, ids, 0.25, softmax=softmax)
    assert (out.mean_probs.double() * E - 1).abs().max().item() <= 2.0 ** -16
    assert abs(out.loss.item() / 0.25 - 1) <= 2.0 ** -15.5
    assert torch.equal(out.counts[0].long(), torch.bincount(ids.flatten(), minlength=E))


def test_the_loss_of_many_sequences():
    # one token each, all to the same experts: 8192 equal terms a thread, whose plain sum is off by
    # 1.2e-4.  Against the loss of the
    # call's own counts and means: a term is two roundings and the sum 1 + 31 + 10 additions of
    # 2^-24 after the compensated one, the scale three more: 2^-18.
    T = S = 65536
    E, K = 4091, 32
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    ids = torch.arange(K, dtype=torch.int32, device=DEV).repeat(T, 1)
    off = torch.arange(T + 1, dtype=torch.int32, device=DEV)
    out = mrs.balance_loss(logits, ids, 1.0, seq_offsets=off)
    want = (out.counts[:, :K].double() * out.mean_probs[:, :K].double()).sum() * (E / K / S)
    assert int(out.counts.sum()) == T * K and int(out.counts[:, :K].min()) == 1
    assert abs(out.loss.item() - want.item()) <= 2.0 ** -18 * want.item()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("weights,loss", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("E,K", [(64, 6), (129, 5), (896, 16), (2056, 8)])
def test_gradients_of_sigmoids_near_one(E, K, weights, loss, dtype):
    # 1 - s, which both terms carry, is e^-17 at a logit of 17: half a step of an s near 1.
    # Relative to |p (1 - s)| (|g| + sum p |g|) and the like of the weights: s is within 2^-23, and
    # 1 - s at least 2^-11 where it is taken from s (2^-12); where it is s e^-x, an argument of 60
    # rounded by 2^-18 and then 2^-21; all else below 2^-15.
    T, R, coef = 200, 2.5, 0.5
    g = torch.Generator().manual_seed(E)
    logits = (24 * torch.rand(T, E, generator=g) + 12 * torch.rand(T, 1, generator=g) - 4).bfloat16()
    logits[1] += 20
    ids = torch.rand(T, E, generator=g).topk(K, dim=1).indices.int()
    gw = torch.randn(T, K, generator=g)
    counts = torch.bincount(ids.flatten().long(), minlength=E).int()[None]
    got = mrs.route_backward(logits.to(DEV), ids.to(DEV), gw.to(DEV) if weights else None, R,
                             grad_loss=torch.ones(1, device=DEV) if loss else None,
                             counts=counts.to(DEV), coef=coef, dtype=dtype).double().cpu()
    x = logits.double()
    s, less = 1 / (1 + (-x).exp()), 1 / (1 + x.exp())
    want, scale = torch.zeros_like(x), torch.zeros_like(x)
    if loss:
        p = s / s.sum(1, keepdim=True)
        f = coef * E / (K * T * T) * counts.double()
        dot = (p * f).sum(1, keepdim=True)
        want += p * less * (f - dot)
        scale += p * less * (f + dot)
    if weights:
        at = ids.long()
        q = s.gather(1, at) / s.gather(1, at).sum(1, keepdim=True)
        c, w = less.gather(1, at), gw.double()
        want.scatter_add_(1, at, R * q * c * (w - (q * w).sum(1, keepdim=True)))
        scale.scatter_add_(1, at, R * q * c * (w.abs() + (q * w.abs()).sum(1, keepdim=True)))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    err = (got - want).abs()
    assert torch.all(err <= 2.0 ** -11.5 * scale + half * want.abs() + 1e-36), (err / scale).max()


GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                    dtype=torch.float64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_scale_byte_with_every_code(dtype):
    # 2^(byte - 127) times the grid, exactly; beyond the type an infinity, byte 255 NaN
    byte = torch.arange(256, dtype=torch.uint8)
    code = torch.arange(32, dtype=torch.uint8) % 16
    codes = (code[0::2] | (code[1::2] << 4)).repeat(256, 1)
    scales = torch.zeros(256, 4, dtype=torch.uint8)
    scales[:, 0] = byte
    got = mrs.mxfp4_dequantize(mrs.Mxfp4Rows(codes.to(DEV), scales.to(DEV)), dtype=dtype).cpu()
    want = torch.pow(2.0, byte.double() - 127)[:, None] * GRID.repeat(2)
    want[255] = float("nan")
    far = want.abs() > torch.finfo(dtype).max
    # 2, 3, 4, 6 of byte 254 and 4, 6 of 253, either sign, each code twice in a block
    assert int(far.sum()) == (4 + 2) * 2 * 2
    want[far] = want[far].sign() * float("inf")
    assert torch.equal(got.double().nan_to_num(7.0, 8.0, -8.0), want.nan_to_num(7.0, 8.0, -8.0))
    assert torch.equal(torch.signbit(got[:255]), torch.signbit(GRID.repeat(2)).expand(255, 32))


def test_products_of_the_furthest_scales():
    # the largest and smallest scale bytes of rows against weights that bring the product back into
    # fp32: exact values (a single product per sum), whatever either factor is by itself
    T, E, K, cols, N, B = 16, 1, 1, 64, 16, 16
    x, w, lists = _layer(T, E, K, cols, N, B)
    x.codes.zero_()
    w.codes.zero_()
    x.codes[:, 0] = 7  # 6 in the first column
    w.codes[0, :, 0] = torch.arange(16, dtype=torch.uint8, device=DEV)  # every code
    for xb, wb in [(254, 20), (254, 120), (253, 100), (252, 127), (20, 254), (0, 200), (0, 254),
                   (1, 252), (100, 30), (127, 254)]:
        x.scales.fill_(xb)
        w.scales.fill_(wb)
        got = mrs.experts_mxfp4(x, w, T, K, B, *lists, dtype=torch.float32).double().cpu()
        want = 6.0 * 2.0 ** (xb + wb - 254) * GRID
        far = want.abs() > torch.finfo(torch.float32).max
        want[far] = want[far].sign() * float("inf")
        assert torch.equal(got, want.expand(T, N)), (xb, wb, got[0], want)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,K", [(64, 1), (376, 1), (129, 5), (896, 16), (2056, 32)])
def test_gradients_of_a_route_that_holds_nearly_all(E, K, softmax):
    # w_k = R q_k and sum q = 1: a token's only route has no gradient, and where one of several has
    # nearly all the weight its gradient is what the others hold.  Relative to
    # R q (|g - g_top| + sum q |g - g_top|): q is within 2^-21 + 30 * 2^-23 and sums are 5 deep: 2^-17
    # (and 2^-12 of 1 - s, as above).
    T, R = 300, 2.5
    g = torch.Generator().manual_seed(E + K)
    logits = (1.5 * torch.randn(T, E, generator=g) - 14).bfloat16()
    ids = torch.rand(T, E, generator=g).topk(K, dim=1).indices.int()
    top = torch.randint(0, K, (T, 1), generator=g)
    lift = 20 * torch.rand(T, 1, generator=g)  # up to e^20 times the others' weights
    logits.scatter_(1, ids.long().gather(1, top), (lift - 14).bfloat16())
    gw = torch.randn(T, K, generator=g)
    got = mrs.route_backward(logits.to(DEV), ids.to(DEV), gw.to(DEV), R, softmax,
                             dtype=torch.float32).double().cpu()
    x = logits.double().gather(1, ids.long())
    u = (x - x.amax(1, keepdim=True)).exp() if softmax else 1 / (1 + (-x).exp())
    q = u / u.sum(1, keepdim=True)
    less = 1.0 if softmax else 1 / (1 + x.exp())
    d = gw.double() - gw.double().gather(1, x.argmax(1, keepdim=True))
    want = R * q * less * (d - (q * d).sum(1, keepdim=True))
    scale = R * q * less * (d.abs() + (q * d.abs()).sum(1, keepdim=True))
    err = (got.gather(1, ids.long()) - want).abs()
    assert torch.all(err <= (2.0 ** -17 + (0 if softmax else 2.0 ** -12)) * scale), \
        (err / scale.clamp(min=1e-300)).max()
    if K == 1:
        assert not got.any()


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,K", [(64, 8), (129, 5), (896, 16), (2056, 8)])
def test_the_loss_gradient_of_an_almost_even_router(E, K, softmax):
    # counts that differ by one in a hundred and more: the gradient p (g - sum p g) lives in those
    # ones.  Relative to p (|g - g0| + sum p |g - g0|), g0 an even router's: a probability is within
    # 2^-18 (as in the other gradient tests) and sum p within 2^-21 of 1, times at most one count;
    # with a sigmoid 1 - s, at least 2^-11 where it is taken from an s within 2^-23: 2^-12.
    T = 200 * E // K
    logits, ids = _router(T, E, K, seed=E)
    g = torch.Generator().manual_seed(E)
    counts = (T * K // E + torch.randint(-1, 2, (1, E), generator=g)).int()
    assert int(counts.min()) >= 198
    got = mrs.route_backward(logits, ids, softmax=softmax, grad_loss=torch.ones(1, device=DEV),
                             counts=counts.to(DEV), coef=0.5, dtype=torch.float32)
    x = logits.double()
    s = torch.softmax(x, 1) if softmax else torch.sigmoid(x)
    p = s / s.sum(1, keepdim=True)
    c = (counts.to(DEV).double() - T * K / E) * (0.5 * E / K / T / T)
    less = 1.0 if softmax else 1 / (1 + x.exp())
    dot = (p * c).sum(1, keepdim=True)
    scale = p * less * (c.abs() + (p * c.abs()).sum(1, keepdim=True))
    assert torch.all((got.double() - p * less * (c - dot)).abs()
                     <= (2.0 ** -17 + (0 if softmax else 2.0 ** -12)) * scale)
    # an even one has nothing to learn
    even = torch.full_like(counts, 200).to(DEV)
    none = mrs.route_backward(logits, ids, softmax=softmax, grad_loss=torch.ones(1, device=DEV),
                              counts=even, coef=0.5, dtype=torch.float32)
    assert none.abs().max().item() <= 2.0 ** -20 * 0.5 / T


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E", [4096, 4095])
def test_router_rows_past_32_bit_offsets(E, softmax):
    # more than 2^31 logits: the last sequence against the same tokens in a call of their own (the
    # CTAs' ranges differ, and with them the order of the column sums)
    T, K, n = 525_000, 4, 1000
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    last, ids = _router(n, E, K)
    logits[-n:] = last
    all_ids = torch.zeros(T, K, dtype=torch.int32, device=DEV)
    all_ids[-n:] = ids
    off = torch.tensor([0, T - n, T], dtype=torch.int32, device=DEV)
    big = mrs.balance_loss(logits, all_ids, 1.0, softmax=softmax, seq_offsets=off)
    one = mrs.balance_loss(last, ids, 1.0, softmax=softmax)
    assert torch.equal(big.counts[1], one.counts[0]) and int(big.counts[0, 0]) == (T - n) * K
    assert torch.all((big.mean_probs[1] - one.mean_probs[0]).abs() <= 2.0 ** -18 * one.mean_probs[0])
    assert (big.mean_probs[0].double() * E - 1).abs().max().item() <= 2.0 ** -16
    gw = torch.randn(n, K, device=DEV)
    all_gw = torch.zeros(T, K, device=DEV)
    all_gw[-n:] = gw
    gl = torch.ones(1, device=DEV)
    grad = mrs.route_backward(logits, all_ids, all_gw, 2.5, softmax, gl, big.counts, 1.0, off)
    # (two sequences: half the coefficient for each; 0.5 is exact)
    want = mrs.route_backward(last, ids, gw, 2.5, softmax, gl, one.counts, 0.5)
    assert torch.equal(grad[-n:], want)
    assert torch.isfinite(grad[0].float()).all()


def test_products_past_32_bit_offsets():
    # outputs of more than 2^31 elements, and weights of more than 2^32 bytes: rows of the last
    # experts against a call that holds those alone
    T, E, K, cols, N, B = 33000, 8, 4, 32, 16400, 64
    x, w, lists = _layer(T, E, K, cols, N, B)
    out = mrs.experts_mxfp4(x, w, T, K, B, *lists)
    xs, part = mrs.mxfp4_dequantize(x), slice(T - 5, T)
    ids = torch.rand(T, E, generator=torch.Generator().manual_seed(0)).topk(K, dim=1).indices
    wv = mrs.mxfp4_dequantize(w)[ids[part].to(DEV)].double()  # [5, K, N, cols]
    want = torch.einsum("tc,tknc->tkn", xs[part].double(), wv)
    mag = torch.einsum("tc,tknc->tkn", xs[part].double().abs(), wv.abs())
    got = out.view(T, K, N)[part].double()
    tol = cols * 2.0 ** -23 * mag
    assert torch.all((got - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 1e-38)
    del out
    T, E, K, cols, N, B = 40, 1100, 1, 4096, 2048, 16
    codes = torch.randint(0, 256, (E, N, cols // 2), dtype=torch.uint8, device=DEV)
    scales = torch.randint(118, 128, (E, N, cols // 32), dtype=torch.uint8, device=DEV)
    assert codes.numel() > 1 << 32
    x = mrs.mxfp4_quantize(torch.randn(T, cols, device=DEV))
    m = mrs.RouteSortBuffers.allocate(T, E, K, B, device=DEV)

    def call(ids, w, E):
        mrs.moe_sort(ids, torch.ones(T, K, device=DEV), E, B, m.sorted_token_ids, m.sorted_weights,
                     m.expert_ids, m.num_tokens_post_pad, m.workspace)
        return mrs.experts_mxfp4(x, w, T, K, B, m.sorted_token_ids, m.expert_ids,
                                 m.num_tokens_post_pad)

    ids = (torch.arange(T, device=DEV)[:, None] % 4).int()
    few = mrs.Mxfp4Rows(codes[-4:].clone(), scales[-4:].clone())
    want = call(ids, few, 4)
    assert torch.equal(call(ids + (E - 4), mrs.Mxfp4Rows(codes, scales), E), want)


def test_buffers_that_start_between_vectors():
    # 4-byte alignment is all that counts, ids, gradients and weights' scales have to have
    T, E, K = 70, 256, 8
    logits, ids = _router(T, E, K)
    gw, gl = torch.randn(T, K, device=DEV), torch.ones(1, device=DEV)
    off = torch.tensor([0, 30, T], dtype=torch.int32, device=DEV)

    def shifted(t):
        room = torch.zeros(t.numel() + 1, dtype=t.dtype, device=DEV)
        room[1:] = t.flatten()
        return room[1:].view(t.shape)

    loss = mrs.balance_loss(logits, ids, 0.5, seq_offsets=off)
    got = [shifted(torch.zeros_like(t)) for t in (loss.loss, loss.counts, loss.mean_probs)]
    mrs.moe_balance_loss(logits, shifted(ids), shifted(off), False, 0.5, *got, loss.workspace)
    assert all(torch.equal(a, b) for a, b in zip(got, (loss.loss, loss.counts, loss.mean_probs)))
    want = mrs.route_backward(logits, ids, gw, 2.5, False, gl, loss.counts, 0.5, off)
    grad = mrs.route_backward(logits, shifted(ids), shifted(gw), 2.5, False, shifted(gl), got[1], 0.5,
                              shifted(off))
    assert torch.equal(grad, want)
    T, E, K, cols, N, B = 20, 4, 2, 512, 136, 16
    x, w, lists = _layer(T, E, K, cols, N, B)
    room = torch.zeros(w.scales.numel() + 4, dtype=torch.uint8, device=DEV)
    room[4:] = w.scales.flatten()
    moved = mrs.Mxfp4Rows(w.codes, room[4:].view(w.scales.shape))
    assert torch.equal(mrs.experts_mxfp4(x, moved, T, K, B, *lists),
                       mrs.experts_mxfp4(x, w, T, K, B, *lists))
