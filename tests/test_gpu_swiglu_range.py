"""The gated activation where sigmoid(a) by itself is smaller than any fp32 number and its product with
a large b, or with a large gradient, is not.

exp(a / 2) is taken once and multiplied twice: an error of 2 + 1.173 |a| / 2 units of 2^-23 each time
(2 for 2^x, and the error of x = a log2(e) / 2, two roundings, times log(2)), a rounding of 2^-24 for each of at most 16 other operations, and
half a step of the result, 2^-8 of it in bf16, 2^-134 where it is subnormal.  exp(a / 2) is a normal
number down to a = -174.
"""
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


def _gates():
    return torch.tensor([-20.0, -60, -80, -87.5, -89, -95, -100, -103, -104, -105, -110, -128, -150,
                         -170], device=DEV).to(BF)


def _slack(a):
    return 2 * (2 + 1.173 * a.abs() / 2) * 2.0**-23 + 16 * 2.0**-24


def _close(got, want, a):
    slack = _slack(a)
    room = (slack + 2.0**-8 * (1 + slack)) * want.abs() + 2.0**-134
    err = (got.double() - want).abs()
    assert (err <= room).all(), (a[err > room], got[err > room], want[err > room])


@pytest.mark.parametrize("rows", [1, 400])  # one and two vectors a thread
@pytest.mark.parametrize("b", [1.0, 2.0**40, -2.0**100, 2.0**120])
def test_forward(rows, b):
    a = _gates()
    cols = 3000
    x = torch.zeros(a.numel() * rows, 2 * cols, dtype=BF, device=DEV)
    x[:, :cols] = a.repeat(rows)[:, None]
    x[:, cols:] = b
    ad = a.double()
    want = ad * torch.sigmoid(ad) * b
    y = mrs.swiglu(x)
    assert (y == y[:, :1]).all()
    _close(y[:, 0], want.repeat(rows), ad.repeat(rows))
    # in 8 bits: all of a row alike, so that each is 448 times the scale, one more rounding each
    q = mrs.swiglu(x, fp8=True)
    got = (q.codes[:, 0].double() * q.scales.double()).view(rows, -1)
    big = want.abs() >= 448 * 2.0**-126
    slack = _slack(ad[big]) + 2 * 2.0**-24
    assert ((got[:, big] - want[big]).abs() <= slack * want[big].abs()).all()


@pytest.mark.parametrize("d,b", [(1.0, 2.0**100), (2.0**100, 1.0), (-2.0**60, 2.0**60)])
def test_backward(d, b):
    a = _gates()
    n = a.numel()
    x = torch.zeros(n, 16, dtype=BF, device=DEV)
    x[:, :8], x[:, 8:] = a[:, None], b
    grad = torch.full((n, 8), d, dtype=BF, device=DEV)
    w = torch.full((n,), 0.5, device=DEV)
    gx, gw = mrs.swiglu_backward(grad, x, w)
    ad = a.double()
    up, down = torch.sigmoid(ad), torch.sigmoid(-ad)
    _close(gx[:, 0], 0.5 * d * b * up * (1 + ad * down), ad)
    _close(gx[:, 8], 0.5 * d * ad * up, ad)
    want = 8 * d * b * ad * up
    assert ((gw.double() - want).abs() <= (_slack(ad) + 8 * 2.0**-24) * want.abs() + 2.0**-146).all()
