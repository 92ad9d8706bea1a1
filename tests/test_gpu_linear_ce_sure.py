"""linear_cross_entropy of rows whose target is nearly sure: a loss of 1e-15 has its
bits, and so has the target's entry of the gradient, 1 - p.

One unit of each row of hidden is not zero, so a logit is one product x = h w (in
bfloat16 exact, in float32 rounded once: 2^-24) and passes to base 2 by two
roundings (scale log2(e), the product): off by 4 * 2^-24 |x| with the subtraction.
So, for the target's x_t and the others' x, o = sum e^(x - x_t) is off by
8 * 2^-24 max|x| + 2^-21 (the exponentials) + (V / 64 + 24) 2^-24 (the sums), and so is
log(1 + o), relative to itself, with 2^-22 of its own."""
import pytest
import torch

import top_routed_grouped_gb300 as moe

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16
U = {F: 2.0 ** -24, B: 2.0 ** -8}


def rows(dtype, T=64, V=500, most=40.0, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(V, T, generator=g, device="cuda") * 0.05
    at = torch.arange(T, device="cuda")
    t = at * 7 % V
    w[t, at] += 1.0
    h = torch.zeros(T, T, device="cuda")
    h[at, at] = torch.linspace(-most / 4, most, T, device="cuda")
    d = 0.5 + torch.rand(T, generator=g, device="cuda")
    return h.to(dtype), w.to(dtype), t, d


def others(h, w, t):
    x = h.double() @ w.double().t()
    xt = x.gather(1, t[:, None])
    x = (x - xt).scatter(1, t[:, None], float("-inf"))
    return torch.exp(x).sum(1), xt[:, 0], (x + xt).abs().nan_to_num(posinf=0.0).amax(1).maximum(xt[:, 0].abs())


@pytest.mark.parametrize("dtype", [F, B])
def test_small_losses_keep_their_bits(dtype):
    h, w, t, d = rows(dtype)
    o, xt, big = others(h, w, t)
    want = torch.log1p(o)
    assert float(want.min()) < 1e-13 and float(want.max()) > 5
    tol = 8 * 2.0 ** -24 * big + 2.0 ** -21 + (w.shape[0] / 64 + 24) * 2.0 ** -24 + 2.0 ** -22
    loss, lse = moe.linear_cross_entropy(h, w, t)
    step = moe.linear_cross_entropy_step(h, w, t, d, dweight_dtype=F)
    assert torch.equal(loss, step[0])
    off = (loss.double() / want - 1).abs() / tol
    assert float(off.max()) <= 1, (int(off.argmax()), float(loss[off.argmax()]), float(want[off.argmax()]))
    # lse: the largest logit to base 2 and back.  The product in float32, the constants log2(e) and
    # ln 2 and the products with them are rounded by 2^-24 of it each, and lse itself once.
    assert bool(((lse - (xt + want)).abs() <= 2.0 ** -24 * (5 * big + lse.abs()) + tol * want).all())
    # dweight[t_i, i] is the target's entry of row i times h_i, which nothing else touches: the row of
    # hidden over its factor is rounded once in bfloat16.
    at = torch.arange(len(t), device="cuda")
    got, ref = step[2][t, at].double(), -d.double() * (o / (1 + o)) * h[at, at].double()
    tol = tol + U[dtype] * 1.01 + 8 * 2.0 ** -24
    assert bool(((got - ref).abs() <= tol * ref.abs()).all()), float(((got / ref - 1).abs() / tol).max())


@pytest.mark.parametrize("dtype", [F, B])
def test_the_gradient_alone_goes_by_lse(dtype):
    """1 - p to 2^-22 |lse|: lse's rounding, the dot product's and the difference's."""
    h, w, t, d = rows(dtype)
    o, xt, big = others(h, w, t)
    _, lse = moe.linear_cross_entropy(h, w, t)
    dw = moe.linear_cross_entropy_backward(d, lse, h, w, t, dweight_dtype=F)[1]
    at = torch.arange(len(t), device="cuda")
    ref = -d.double() * (o / (1 + o))
    got = dw[t, at].double() / h[at, at].double()
    tol = (2.0 ** -22 * (big + lse.abs()) + 2.0 ** -21) * d + U[dtype] * 1.02 * ref.abs()
    assert bool(((got - ref).abs() <= tol).all()), float(((got - ref).abs() / tol).max())


@pytest.mark.parametrize("dtype", [F, B])
def test_targets_that_are_alone_or_hold_infinity(dtype):
    w = torch.randn(1, 64, device="cuda").to(dtype)  # a vocabulary of one: sure, always
    h = torch.randn(5, 64, device="cuda").to(dtype)
    t, d = torch.zeros(5, dtype=torch.int64, device="cuda"), torch.ones(5, device="cuda")
    loss, dh, dw = moe.linear_cross_entropy_step(h, w, t, d)
    assert not loss.any() and not dh.any() and not dw.any()
    lse = moe.linear_cross_entropy(h, w, t)[1]
    x = (h.double() @ w.double().t())[:, 0]
    assert bool(((lse - x).abs() <= 72 * 2.0 ** -23 * (h.double().abs() @ w.double().abs().t())[:, 0]).all())
    # The target's logit is infinite, or another is: no finite loss; below everything: an infinite one.
    w = torch.zeros(65, 64, device="cuda", dtype=dtype)
    w[:, 0] = 1
    for v, value in ((64, float("inf")), (3, float("inf")), (64, float("-inf"))):
        ww = w.clone()
        ww[v, 0] = value
        loss = moe.linear_cross_entropy(torch.ones_like(h), ww, torch.full_like(t, 64))[0]
        assert not torch.isfinite(loss).any()
    ww = w.clone()
    ww[3, 0] = float("-inf")  # a token that cannot come
    loss = moe.linear_cross_entropy(torch.ones_like(h), ww, torch.full_like(t, 64))[0]
    assert bool(((loss - torch.log(torch.tensor(64.0, dtype=torch.float64))).abs() <= 1e-5).all())
