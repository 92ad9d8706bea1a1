"""linear_cross_entropy in forms that sizes alone bring about: wide rows, float
gradients in several pieces of the vocabulary, many rows with 32-bit targets."""
import pytest
import torch

import top_routed_grouped_gb300 as moe
from _train_ref import IGNORE
from test_gpu_linear_ce import all_ok, make, status

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("T,D,V,dtype", [(300, 4096, 700, B), (37, 4090, 1000, B), (9, 16384, 300, B), (300, 16383, 130, B),
                                         (40, 4096, 200, F), (5, 16384, 70, F)])
def test_wide_rows(T, D, V, dtype):
    all_ok(*make(T, D, V, dtype, left_out=T // 4))


@pytest.mark.parametrize("T,D,V", [(65536, 40, 1300),   # one chunk of 512 columns a piece, added to the sums before
                                   (16384, 64, 4613)])  # two pieces of several chunks
def test_float_in_pieces(T, D, V):
    all_ok(*make(T, D, V, F, left_out=T // 10))


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("T", [4097, 20011])
def test_many_rows_with_targets_of_32_bits(T, dtype):
    h, w, t, d = make(T, 64, 130, dtype, left_out=T // 3)
    for a, b in zip(moe.linear_cross_entropy_step(h, w, t, d), moe.linear_cross_entropy_step(h, w, t.int(), d)):
        assert torch.equal(a, b)
    assert status() == 0
    bad = t.int()
    bad[T - 1], bad[8], bad[4096] = 130, -5, 1 << 30
    want = torch.where((bad >= 0) & (bad < 130), bad, IGNORE)
    got = moe.linear_cross_entropy_step(h, w, bad, d)
    assert status() == 7
    assert all(torch.equal(a, b) for a, b in zip(got, moe.linear_cross_entropy_step(h, w, want, d))) and status() == 0


@pytest.mark.parametrize("D", [2048, 16384])
def test_logits_of_one_sign(D):
    """D addends of one sign that make 60, in chains of 512 of the tensor cores' cut-off sums (2^-23 of a
    sum that is half of the chain's on average, an addend) and an FP32 sum of the chains (2^-24 each): x
    within (512 + D / 512) 2^-24 of itself, and lse with it; 2^-18 for the exponentials and the rest.  One
    chain over D = 16384 is off by twice that."""
    V = 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    h = (0.5 + 0.5 * torch.rand(3, D, generator=g, device="cuda")).to(B)
    w = ((0.5 + 0.5 * torch.rand(V, D, generator=g, device="cuda")) * (60 / (0.5625 * D))).to(B)
    t = torch.tensor([5, 0, V - 1], device="cuda")
    x = h.double() @ w.double().t()
    want = torch.logsumexp(x, 1)
    loss, lse = moe.linear_cross_entropy(h, w, t)
    tol = (512 + D / 512) * 2.0 ** -24 * x.amax(1) + 2.0 ** -18
    print(f"D = {D}: lse {float((lse - want).abs().max()):.1e} off, bound {float(tol.max()):.1e}")
    assert bool(((lse - want).abs() <= tol).all())
    assert bool(((loss - (want - x.gather(1, t[:, None])[:, 0])).abs() <= 2 * tol).all())
