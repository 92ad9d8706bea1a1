"""linear_cross_entropy: long sums keep their bits.

The tensor cores cut an FP32 sum off where others round it, 2^-23 of what it has
come to for an addend at most, so a sum of one sign in one chain is short by an
amount that grows with its length.  The bounds here count the chains that the
operator documents and not the whole sums; inputs are such that nothing else is
rounded where it would show."""
import pytest
import torch

import top_routed_grouped_gb300 as moe

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("T", [8192, 8193, 40000, 1 << 21])
def test_dweight_of_many_rows_on_one_target(T):
    """Logits of 0 over two tokens: g is a power of 2 and dweight its product with
    the sum of hidden, all of one sign.  Chains of 8192 rows, each addend cut off
    by 2^-23 of a sum that is half of the chain's on average: 8192 * 2^-24; the
    chains' own sums rounded: 2^-24 each."""
    g = torch.Generator(device="cuda").manual_seed(1)
    h = (0.5 + 0.5 * torch.rand(T, 64, generator=g, device="cuda")).to(B)
    w = torch.zeros(2, 64, dtype=B, device="cuda")
    t = torch.zeros(T, dtype=torch.int64, device="cuda")
    d = torch.full((T,), 2.0 ** -9, device="cuda")
    want = h.double().sum(0) * 2.0 ** -10
    tol = (min(T, 8192) + T / 8192 + 4) * 2.0 ** -24
    base = torch.randn(2, 64, device="cuda")
    acc = base.clone()
    moe.linear_cross_entropy_step(h, w, t, d, dweight=acc)
    _, lse = moe.linear_cross_entropy(h, w, t)
    for dw in (moe.linear_cross_entropy_step(h, w, t, d, dweight_dtype=F)[2],
               moe.linear_cross_entropy_backward(d, lse, h, w, t, dweight_dtype=F)[1]):
        off = (dw.double() / torch.stack([-want, want]) - 1).abs().max()
        print(f"T = {T}: dweight {float(off):.2e} off, bound {tol:.2e}")
        assert float(off) <= tol
    assert torch.equal(acc, base + dw)


@pytest.mark.parametrize("D", [512, 2048, 4096, 16384])
def test_probabilities_of_a_row_add_up_to_one(D):
    """The gradient's logits are those that the statistics were taken of, to the
    last bit, so that the row of g adds up to 0 however far the logits' sums are
    off, here of D addends of one sign that make 60.  Each entry but the target's
    is rounded to bfloat16, by 2^-8 of it at most: six times the root of the sum
    of those squares (by Hoeffding's bound exceeded once in 10^7), and 2^-18 for
    the exponentials and their sum."""
    V = 8192
    g = torch.Generator(device="cuda").manual_seed(2)
    h = (0.5 + 0.5 * torch.rand(1, D, generator=g, device="cuda")).to(B)
    w = ((0.5 + 0.5 * torch.rand(V, D, generator=g, device="cuda")) * (60 / (0.5625 * D))).to(B)
    t, d = torch.tensor([5], device="cuda"), torch.ones(1, device="cuda")
    x = (w.double() @ h[0].double())
    p = torch.softmax(x, 0)
    assert 50 < float(x.mean()) < 70
    _, lse = moe.linear_cross_entropy(h, w, t)
    for dw in (moe.linear_cross_entropy_step(h, w, t, d, dweight_dtype=F)[2],
               moe.linear_cross_entropy_backward(d, lse, h, w, t, dweight_dtype=F)[1]):
        # dweight's rows are g_v times one and the same rounding of hidden.
        row = dw[5].double()
        gv = (dw.double() @ row) / (row @ row)   # in units of the target's entry
        total = float(gv.sum())
        bound = 6 * 2.0 ** -8 * float(p.square().sum().sqrt()) + 2.0 ** -18
        print(f"D = {D}: a row of g adds up to {total:.2e}, bound {bound:.2e}")
        assert abs(total) <= bound
