"""The balance loss with its counts, and the gradient to the router logits, on a GB300, against a
plain float64 implementation (torch.autograd of the definitions for the gradient).

Tolerances, set by arithmetic: a probability is a product of an exponential within 2^-21 (ex2 of
an argument rounded once, |x| <= 12), a reciprocal within 2^-22 and a sum of up to 4096 terms in
32 lanes times 32 columns (at most 50 additions deep, each 2^-24): below 2^-18 relative.  A mean
over T <= 3000 tokens adds at most T / 8 sequential additions of equal-signed terms a group, whose
rounding is at most 400 * 2^-24 = 2^-15.4 of the sum.  The loss is a weighted mean of them.  A
gradient is a difference g - sum p g: relative to |p| (|g| + sum p |g|), 2^-15.  bf16 outputs add
half a step, 2^-8 of the value, and float32 gradients nothing.
"""
import math

import pytest
import torch

import moe_expert_routing_sort_gb300 as mrs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
REL = 2.0 ** -15


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mrs.build()
    mrs.load()


def _inputs(T, E, K, seed=0, std=1.5, drop=True):
    g = torch.Generator().manual_seed(seed)
    logits = (std * torch.randn(T, E, generator=g)).bfloat16()
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]) if T else \
        torch.zeros(0, K)
    ids = ids.int()
    if drop and T > 3:
        ids[T // 2, 0] = -1
        ids[T // 3, :] = -1
        ids[1, K - 1] = E + 5
    return logits.to(DEV), ids.to(DEV)


def _probs(x, softmax):
    if softmax:
        m = x.amax(1, keepdim=True).clamp(min=-1e300)
        e = (x - m).exp()
        s = e.sum(1, keepdim=True)
        return torch.where(s > 0, e / s, 0.0)
    s = 1 / (1 + (-x).exp())
    z = s.sum(1, keepdim=True)
    return torch.where(z > 0, s / z, 0.0)


def _ref_loss(x, ids, off, E, K, coef, softmax):
    S = len(off) - 1
    loss = torch.zeros((), dtype=torch.float64)
    counts, means = [], []
    for a, b in zip(off[:-1], off[1:]):
        i = ids[a:b].reshape(-1).long()
        c = torch.bincount(i[(i >= 0) & (i < E)], minlength=E)
        m = _probs(x[a:b], softmax).sum(0) / max(b - a, 1)
        loss = loss + coef / S * (c.double() * (E / K) / max(b - a, 1) * m).sum()
        counts.append(c)
        means.append(m)
    return loss, torch.stack(counts), torch.stack(means)


def _check_loss(logits, ids, off, coef, softmax, stream=None, out=None):
    T, E = logits.shape
    K = ids.shape[1]
    d_off = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    out = mrs.balance_loss(logits, ids, coef, softmax=softmax, seq_offsets=d_off, out=out,
                           stream=stream)
    torch.cuda.synchronize()
    loss, counts, means = _ref_loss(logits.double().cpu(), ids.cpu(), off or [0, T], E, K, coef,
                                    softmax)
    assert torch.equal(out.counts.cpu().long(), counts)
    m = out.mean_probs.double().cpu()
    assert torch.all((m - means).abs() <= REL * means + 1e-30)
    assert abs(out.loss.item() - loss.item()) <= REL * abs(loss.item())
    return out


SHAPES = [  # E, K: every load width, columns per lane and warps per row
    (1, 1), (7, 3), (64, 6), (129, 5), (256, 8), (520, 32), (896, 16), (1000, 8), (1031, 4),
    (2056, 8), (2500, 2), (4095, 7), (4096, 32),
]


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("T", [1, 2, 67, 1000])
@pytest.mark.parametrize("E,K", SHAPES)
def test_loss_of_one_sequence(E, K, T, softmax):
    logits, ids = _inputs(T, E, K, seed=E + T)
    _check_loss(logits, ids, None, 0.01, softmax)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("T,off", [
    (300, [0, 300]), (300, [0, 1, 2, 3, 300]), (300, [0, 0, 0, 299, 300]),
    (300, [5, 17, 17, 200, 280]), (3000, [0, 1024, 1025, 2047, 2048, 3000]),
    (2000, list(range(0, 2001, 10))), (40, [40, 40]), (10, [0, 10] + [10] * 60),
])
@pytest.mark.parametrize("E,K", [(64, 6), (129, 5), (2056, 8)])
def test_loss_of_packed_sequences(E, K, T, off, softmax):
    logits, ids = _inputs(T, E, K, seed=len(off))
    _check_loss(logits, ids, off, 0.5, softmax)


def test_borders_outside_the_tokens_act_as_the_ends():
    logits, ids = _inputs(50, 64, 4)
    a = mrs.balance_loss(logits, ids, 1.0, seq_offsets=torch.tensor([-7, 20, 90], dtype=torch.int32,
                                                                    device=DEV))
    b = _check_loss(logits, ids, [0, 20, 50], 1.0, False)
    assert torch.equal(a.loss, b.loss) and torch.equal(a.counts, b.counts)


@pytest.mark.parametrize("softmax", [False, True])
def test_no_tokens(softmax):
    logits, ids = _inputs(0, 64, 4)
    out = mrs.balance_loss(logits, ids, 1.0, softmax=softmax)
    assert out.loss.item() == 0 and not out.counts.any() and not out.mean_probs.any()
    assert mrs.route_backward(logits, ids).shape == (0, 64)


def test_an_even_router_has_loss_coef():
    E, K, T = 64, 8, 64
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    ids = ((torch.arange(T)[:, None] + torch.arange(K)) % E).int().to(DEV)
    for softmax in (False, True):
        out = _check_loss(logits, ids, None, 0.25, softmax)
        assert abs(out.loss.item() - 0.25) <= REL


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E", [129, 896, 2056])
def test_masked_experts(E, softmax):
    # -inf logits: masked experts, a token with one expert left, a token with none; the type's
    # lowest and highest values
    logits, ids = _inputs(40, E, 4)
    logits[:, ::3] = -math.inf
    logits[3, :] = -math.inf
    logits[3, 7] = 1.0
    logits[4, :] = -math.inf
    logits[5, :] = torch.finfo(torch.bfloat16).min
    logits[6, 1] = torch.finfo(torch.bfloat16).max
    if not softmax:
        logits[5] = -3.0
    out = _check_loss(logits, ids, None, 1.0, softmax)
    assert torch.isfinite(out.mean_probs).all()
    gw = torch.randn(40, 4, device=DEV)
    grad = mrs.route_backward(logits, ids, gw, 2.5, softmax, grad_loss=torch.ones(1, device=DEV),
                              counts=out.counts, coef=1.0, dtype=torch.float32)
    assert torch.isfinite(grad).all()
    assert not grad[logits == -math.inf].any()


def _ref_grad(logits, ids, gw, R, softmax, gl, counts, off, coef):
    """Gradient in float64 by autograd, and the magnitude its rounding errors scale with."""
    x = logits.double().cpu().requires_grad_()
    T, E = x.shape
    K = ids.shape[1]
    total = (x * 0).sum()
    scale = torch.zeros(T, E, dtype=torch.float64)
    if gl is not None:
        S = len(off) - 1
        p = _probs(x, softmax)
        for i, (a, b) in enumerate(zip(off[:-1], off[1:])):
            if b > a:
                g = gl * coef / S * E / (K * (b - a) ** 2) * counts[i].double().cpu()
                total = total + (p[a:b] * g).sum()
                pd = p[a:b].detach()
                scale[a:b] += pd * (g + (pd * g).sum(1, keepdim=True))
    if gw is not None:
        i = ids.cpu().long()
        fine = (i >= 0) & (i < E)
        at = torch.where(fine, i, 0)
        xk = x.gather(1, at)
        u = torch.exp(xk - x.detach().amax(1, keepdim=True)) if softmax else 1 / (1 + (-xk).exp())
        u = u * fine
        z = u.sum(1, keepdim=True)
        w = R * u / torch.where(z > 0, z, 1.0)
        g = gw.double().cpu() * fine
        total = total + (w * g).sum()
        wd = w.detach()
        m = (wd * g.abs()).sum(1, keepdim=True) / max(R, 1e-30)
        scale.scatter_add_(1, at, wd * (g.abs() + m) * fine)
    return torch.autograd.grad(total, x)[0], scale


def _check_grad(logits, ids, off, softmax, dtype, weights=True, loss=True, R=2.5, seed=1):
    T, E = logits.shape
    K = ids.shape[1]
    g = torch.Generator().manual_seed(seed)
    gw = torch.randn(T, K, generator=g).to(DEV) if weights else None
    gl = torch.tensor([0.75], device=DEV) if loss else None
    d_off = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    counts = mrs.balance_loss(logits, ids, 0.5, softmax=softmax, seq_offsets=d_off).counts
    out = torch.full((T, E), float("nan"), dtype=dtype, device=DEV)
    mrs.route_backward(logits, ids, gw, R, softmax, gl, counts if loss else None, 0.5, d_off,
                       out=out)
    torch.cuda.synchronize()
    ref, scale = _ref_grad(logits, ids, gw, R, softmax, 0.75 if loss else None, counts,
                           off or [0, T], 0.5)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    err = (out.double().cpu() - ref).abs()
    assert torch.all(err <= REL * scale + half * ref.abs() + 1e-30), (err - REL * scale).max()
    return out, ref


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("T", [1, 33, 700])
@pytest.mark.parametrize("E,K", SHAPES)
def test_gradient(E, K, T, softmax, dtype):
    logits, ids = _inputs(T, E, K, seed=E + T)
    _check_grad(logits, ids, None, softmax, dtype)


@pytest.mark.parametrize("weights,loss", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("softmax", [False, True])
def test_gradient_of_either_term(softmax, weights, loss):
    logits, ids = _inputs(200, 896, 16)
    out, ref = _check_grad(logits, ids, None, softmax, torch.float32, weights, loss)
    if not weights and not loss:
        assert not out.any()


@pytest.mark.parametrize("weights,loss", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("softmax,shift", [(True, 200.0), (True, -200.0), (True, 5000.0),
                                           (False, 60.0), (False, -60.0)])
def test_gradient_far_from_zero(softmax, shift, weights, loss):
    # e^200 is no fp32 number; a softmax only knows differences, and e^-60 is one
    logits, ids = _inputs(200, 129, 5)
    logits = (logits.float() + shift).bfloat16()
    _check_grad(logits, ids, None, softmax, torch.float32, weights, loss)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("T,off", [
    (300, [0, 1, 2, 3, 300]), (300, [5, 17, 17, 200, 280]), (300, [0, 0, 0, 299, 300]),
    (2000, list(range(0, 2001, 10))), (40, [40, 40]),
])
@pytest.mark.parametrize("E,K", [(64, 6), (129, 5), (2056, 8)])
def test_gradient_of_packed_sequences(E, K, T, off, softmax):
    logits, ids = _inputs(T, E, K, seed=len(off))
    _check_grad(logits, ids, off, softmax, torch.float32)


@pytest.mark.parametrize("softmax", [False, True])
def test_an_expert_named_twice(softmax):
    logits, ids = _inputs(64, 64, 6, drop=False)
    ids[:, 3] = ids[:, 0]
    ids[::2, 5] = ids[::2, 0]
    _check_grad(logits, ids, None, softmax, torch.float32)


@pytest.mark.parametrize("softmax", [False, True])
def test_gradient_against_differences(softmax):
    # the loss's own value moves by the gradient times a step: two bf16 neighbours of a logit
    T, E, K = 8, 64, 6
    logits, ids = _inputs(T, E, K, drop=False)
    logits = (logits.float().clamp(-2, 2) * 8).round().div(8).bfloat16()
    out = mrs.balance_loss(logits, ids, 64.0, softmax=softmax)
    grad = mrs.route_backward(logits, ids, None, 1.0, softmax, torch.ones(1, device=DEV),
                              out.counts, 64.0, dtype=torch.float32)
    for t, e in [(0, int(ids[0, 0])), (3, 5), (7, int(ids[7, 2]))]:
        h, at = 2.0 ** -4, logits[t, e].clone()
        two = []
        for sgn in (1, -1):
            moved = logits.clone()
            moved[t, e] = at + sgn * h
            two.append(mrs.balance_loss(moved, ids, 64.0, softmax=softmax).loss.double().item())
        slope = (two[0] - two[1]) / (2 * h)
        # third derivative of a probability is at most 1 (times 64 E c / (K T^2) <= 64 * 64 / 48);
        # float32 losses near 64 are within 2^-18 * 64
        tol = h * h / 6 * 64 * 64 / 48 * 0.1 + 2 ** -12 / h
        assert abs(slope - grad[t, e].item()) <= tol


def test_gradients_of_the_weights_match_the_route_step():
    # the weights that moe_topk returns are those the gradient is taken of
    T, E, K, R = 64, 256, 8, 2.5
    logits, _ = _inputs(T, E, K, drop=False)
    bias = torch.zeros(E, device=DEV)
    out = mrs.route_sort(logits, bias, 8, 4, K, R, 16)
    x = logits.double().cpu().requires_grad_()
    u = torch.sigmoid(x).gather(1, out.topk_ids.long().cpu())
    w = R * u / u.sum(1, keepdim=True)
    assert (w.detach() - out.topk_weights.double().cpu()).abs().max() <= 1e-6
    gw = torch.randn(T, K, generator=torch.Generator().manual_seed(2))
    ref = torch.autograd.grad((w * gw).sum(), x)[0]
    got = mrs.route_backward(logits, out.topk_ids, gw.to(DEV), R, dtype=torch.float32)
    assert (got.double().cpu() - ref).abs().max() <= REL * R * gw.abs().max()


def test_same_bits_every_call_and_any_workspace():
    logits, ids = _inputs(5000, 896, 16)
    off = torch.tensor([0, 700, 701, 4000, 4900], dtype=torch.int32, device=DEV)
    buf = mrs.BalanceBuffers.allocate(5000, 896, 4, device=DEV)
    buf.workspace.fill_(0xA5)
    a = mrs.balance_loss(logits, ids, 0.1, seq_offsets=off, out=buf)
    first = [t.clone() for t in (a.loss, a.counts, a.mean_probs)]
    buf.workspace.fill_(0xFF)
    for _ in range(3):
        a = mrs.balance_loss(logits, ids, 0.1, seq_offsets=off, out=buf)
        assert all(torch.equal(p, q) for p, q in zip(first, (a.loss, a.counts, a.mean_probs)))


def test_captured_graph_and_other_stream():
    logits, ids = _inputs(400, 896, 16)
    gw = torch.randn(400, 16, device=DEV)
    gl = torch.ones(1, device=DEV)
    buf = mrs.BalanceBuffers.allocate(400, 896, device=DEV)
    grad = torch.empty(400, 896, dtype=torch.bfloat16, device=DEV)

    def step():
        mrs.balance_loss(logits, ids, 0.1, out=buf)
        mrs.route_backward(logits, ids, gw, 2.5, False, gl, buf.counts, 0.1, out=grad)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    fresh, fids = _inputs(400, 896, 16, seed=9)
    logits.copy_(fresh)
    ids.copy_(fids)
    graph.replay()
    torch.cuda.synchronize()
    got = (buf.loss.clone(), buf.counts.clone(), grad.clone())
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (buf.loss, buf.counts, grad)))
    _check_loss(logits, ids, None, 0.1, False)


def test_outputs_stay_inside_their_buffers():
    # canaries around every output at exactly the documented lengths
    for T, E, K, S in [(37, 129, 5, 3), (64, 896, 16, 2), (5, 4095, 3, 4), (9, 1, 1, 1)]:
        logits, ids = _inputs(T, E, K)
        off = torch.linspace(0, T, S + 1).int().to(DEV)
        ws = mrs.moe_balance_workspace_bytes(T, E, S)

        def guarded(n, dtype):
            size = torch.empty(0, dtype=dtype).element_size()
            raw = torch.full((n * size + 2048,), 0x5A, dtype=torch.uint8, device=DEV)
            return raw, raw[1024:1024 + n * size].view(dtype)

        bufs = {k: guarded(n, d) for k, (n, d) in dict(
            loss=(1, torch.float32), counts=(S * E, torch.int32), mean=(S * E, torch.float32),
            ws=(ws, torch.uint8), grad=(T * E, torch.bfloat16)).items()}
        v = {k: b[1] for k, b in bufs.items()}
        mrs.moe_balance_loss(logits, ids, off, True, 1.0, v["loss"], v["counts"], v["mean"], v["ws"])
        mrs.moe_route_backward(logits, ids, None, v["loss"], v["counts"], off, True, 1.0, 1.0,
                               v["grad"])
        torch.cuda.synchronize()
        for k, (raw, view) in bufs.items():
            n = view.numel() * view.element_size()
            assert (raw[:1024] == 0x5A).all() and (raw[1024 + n:] == 0x5A).all(), k


def test_a_call_on_another_stream_makes_its_buffers_there():
    logits, ids = _inputs(300, 129, 5)
    gw = torch.randn(300, 5, device=DEV)
    want = mrs.balance_loss(logits, ids, 0.1)
    grad = mrs.route_backward(logits, ids, gw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        torch.cuda._sleep(50_000_000)
        got = mrs.balance_loss(logits, ids, 0.1, stream=stream)
        got_grad = mrs.route_backward(logits, ids, gw, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got.loss, want.loss) and torch.equal(got.counts, want.counts)
        assert torch.equal(got_grad, grad)
