"""distill over many rows, in each of its modes, to bounds near its roundings.

With u = 2^-24, tau the temperature, x = teacher / tau, c its normaliser, and
size = max |z| / tau + |lse| of a row:

  lse      its terms' exponents are off by a few u of |z| / tau (the factor
           1 / tau and its product with log2 e are rounded once each, the
           exponent once, exp2 by two units), which is u (8 size) of the sum; a
           sum of positive terms adds one u for each addition on a term's way: 64
           in a thread, 5 in a warp, 16 over warps, 8 over CTAs, 8 over passes,
           each join with a power of its own: below 256.  What the logarithm
           and its sum with m / tau round is within 8 size, too.
  loss     sum_k p_k (x_k - c - (z_k / tau - lse)): each p_k is off by
           u (16 + 4 (|x_k| + |c|)) of itself, the difference by 8 u (|x_k| +
           |c| + |z_k| / tau + |lse|) and by lse's own error.
  dlogits  w s / tau (P q - p): q is off by u (256 + 16 size) of itself, by the
           same once more where it comes from a stored lse, whose error it
           has; p as above.  Then half an ulp of the type.
"""
import pytest
import torch

import top_routed_grouped_gb300 as moe

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24
HALF_ULP = {F32: U, BF16: 2.0 ** -8}


def off_by(got, want, bound, what):
    e = (got.double() - want).abs()
    bad = ~(e <= bound)
    if bad.any():
        i = int((e / bound.clamp_min(1e-300)).flatten().argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {e.numel()} off, worst at {i}: {got.flatten()[i]} for "
                             f"{want.flatten()[i]}, bound {bound.flatten()[i]}")


def hold(z, ids, t, w, tau, loss=None, lse=None, grads=(), scale=1.0):
    """Holds what is given to the bounds above, some rows at a time.  grads:
    pairs of dlogits and whether they come from a stored lse."""
    n = max(1, (1 << 25) // z.shape[1])
    for a in range(0, z.shape[0], n):
        i = slice(a, a + n)
        y, x = z[i].double() / tau, t[i].double() / tau
        m = y.abs().amax(1)
        c, l = torch.logsumexp(x, 1), torch.logsumexp(y, 1)
        size = m + l.abs()
        p = torch.softmax(x, 1)
        p_off = p * (16 + 4 * (x.abs() + c.abs()[:, None])) * U
        l_off = (256 + 8 * size) * U
        at = ids[i].long()
        yk = y.gather(1, at)
        d = x - c[:, None] - (yk - l[:, None])
        if lse is not None:
            off_by(lse[i], l, l_off, "lse")
        if loss is not None:
            d_off = 8 * U * (x.abs() + c.abs()[:, None] + yk.abs() + l.abs()[:, None]) + l_off[:, None]
            off_by(loss[i], scale * (p * d).sum(1), abs(scale) * (p_off * d.abs() + p * d_off).sum(1), "loss")
        k = (w[i].double() * scale / tau)[:, None]
        q = torch.exp(y - l[:, None])
        want = (q * k).scatter_add(1, at, -p * k)
        for g, stored in grads:
            q_off = (256 + 16 * size[:, None]) * (2 if stored else 1) * U
            bound = ((q * q_off).scatter_add(1, at, p_off + 4 * U * p) * k.abs() + 4 * U * want.abs()) * (1 + HALF_ULP[z.dtype])
            off_by(g[i], want, bound + HALF_ULP[z.dtype] * want.abs() + 1e-37, "dlogits")


def place(rows, ld, at):
    """Rows as a window of a buffer of NaN, and the buffer."""
    T, V = rows.shape
    buf = torch.full((at + T * ld + 16,), float("nan"), device="cuda", dtype=rows.dtype)
    view = buf.as_strided((T, V), (ld, 1), at)
    view.copy_(rows)
    return view, buf


def beside(buf, T, V, ld, at):
    """What the buffer holds beside the rows."""
    b = buf.clone()
    b.as_strided((T, V), (ld, 1), at).fill_(float("nan"))
    return b


def make(T, V, K, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + T + V + K)
    z = (3 * torch.randn(T, V, generator=g, device="cuda")).to(dtype)
    part = V // K
    ids = torch.arange(K, device="cuda") * part + torch.randint(part, (T, K), generator=g, device="cuda")
    return z, ids.int(), 2 * torch.randn(T, K, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")


@pytest.mark.parametrize("dtype,T,V", [(F32, 3000, 1000), (BF16, 3000, 1003), (F32, 1500, 5003), (BF16, 1500, 8200), (F32, 1500, 16384),
                                       (BF16, 1200, 12000), (BF16, 1200, 16001), (F32, 700, 32000), (BF16, 900, 32000), (F32, 400, 50257),
                                       (BF16, 700, 50257), (F32, 400, 100000), (BF16, 400, 131072), (F32, 300, 131072), (BF16, 200, 262144),
                                       (F32, 60, 300001), (BF16, 60, 524300)])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_many_rows_in_each_mode(dtype, T, V, tau):
    """Each cluster walks over a number of rows, with loss and gradient alone, too."""
    z, ids, t, w = make(T, V, 8, dtype)
    loss, lse = moe.distill(z, ids, t, tau, 1.5)
    hold(z, ids, t, w, tau, loss, lse, scale=1.5)
    step, d2 = moe.distill_step(z, ids, t, w, tau, 1.5)
    hold(z, ids, t, w, tau, step, None, [(d2, False)], scale=1.5)
    hold(z, ids, t, w, tau, grads=[(moe.distill_backward(w, lse, z, ids, t, tau, 1.5), True)], scale=1.5)


def places(V, N):
    """Both sides of every 32nd 16-byte unit, of the shares of up to 8 CTAs,
    of the ends, and some in between."""
    units = -(-V // N)
    at = [u * N for u in range(0, units, 32)]
    at += [-(-n // c) * i * N for n in (units, units + 1) for c in (2, 4, 8) for i in range(c + 1)]
    at += list(range(0, 2 * N)) + list(range(V - 2 * N, V)) + list(range(V // 3, V // 3 + 2 * N))
    return sorted({p + d for p in at for d in (-N, -1, 0, 1, N - 1) if 0 <= p + d < V})


@pytest.mark.parametrize("V,ld,at,ld_out,at_out", [
    (1000, 1000, 0, 1000, 0), (1003, 1003, 0, 1003, 3), (999, 1003, 1, 1002, 4), (8184, 8184, 0, 8184, 0), (8189, 8189, 5, 8190, 2),
    (16000, 16000, 0, 16000, 0), (16001, 16001, 0, 16001, 0), (16001, 16001, 2, 16004, 0), (16384, 16385, 1, 16384, 0), (32000, 32003, 0, 32008, 5),
    (50257, 50257, 0, 50257, 0), (50257, 50257, 0, 50257, 7), (50264, 50264, 0, 50266, 0), (65536, 65536, 0, 65536, 0), (131072, 131072, 0, 131073, 1),
    (100001, 100001, 6, 100008, 0), (300001, 300001, 0, 300003, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_place_of_a_row_is_lost(dtype, V, ld, at, ld_out, at_out):
    """One logit that outweighs its row, in turn at every place where a unit, a
    warp's or a CTA's share or an aligned piece may end: without it, or with
    it twice, lse is off by 0.7 or more.  Logits and gradient start at
    different places; nothing is written beside the rows."""
    where = places(V, 16 // dtype.itemsize)
    keep = max(1, len(where) * V // (1 << 28) + 1)  # (of long rows every few, the first and last ones always)
    where = torch.tensor(where[:40] + where[40:-40][::keep] + where[-40:], device="cuda")
    T = len(where)
    z, ids, t, w = make(T, V, 3, dtype)
    z = (z.float() * 0.25).to(dtype)
    z.scatter_(1, where[:, None], 25.0)
    ids[::2, 1] = where[::2].int()  # a teacher's token in half of the rows
    rows, _ = place(z, ld, at)
    loss, lse = moe.distill(rows, ids, t)
    hold(z, ids, t, w, 1.0, loss, lse)
    for stored in (False, True):
        out, buf = place(torch.zeros_like(z), ld_out, at_out)
        if stored:
            d = moe.distill_backward(w, lse, rows, ids, t, out=out)
        else:
            step, d = moe.distill_step(rows, ids, t, w, out=out)
            hold(z, ids, t, w, 1.0, step)
        assert d is out
        hold(z, ids, t, w, 1.0, grads=[(d, stored)])
        assert torch.isnan(beside(buf, T, V, ld_out, at_out)).all()
    inplace, buf = place(z, ld, at)
    moe.distill_step(inplace, ids, t, w, out=inplace)
    hold(z, ids, t, w, 1.0, grads=[(inplace, False)])
    assert torch.isnan(beside(buf, T, V, ld, at)).all()


@pytest.mark.parametrize("V", [1000, 16001, 32000, 50257, 300001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step_that_leaves_lse(dtype, V):
    """The C entry point writes lse where it is asked to: of rows without a
    teacher or of weight 0, too, which the step need not read otherwise; loss
    and gradient are the same bits."""
    from top_routed_grouped_gb300 import step
    z, ids, t, w = make(300, V, 4, dtype)
    ids[::3], w[::5] = -1, 0
    loss, d = moe.distill_step(z, ids, t, w)
    loss2, lse, d2 = torch.empty_like(loss), torch.empty_like(loss), torch.empty_like(d)
    step.moe_distill_step(step._DISTILL.pack(300, V, 4, step._DTYPE[dtype], 1.0, 1.0, 0, 0, z.data_ptr(), ids.data_ptr(), t.data_ptr(), 0,
                                             w.data_ptr(), loss2.data_ptr(), lse.data_ptr(), d2.data_ptr()),
                          torch.cuda.current_stream().cuda_stream)
    assert torch.equal(loss2, loss) and torch.equal(d2, d)
    assert not loss[::3].any() and not d[::3].any() and not d[::5].any()
    y = z.double()
    off_by(lse, torch.logsumexp(y, 1), U * (256 + 8 * (y.abs().amax(1) + torch.logsumexp(y, 1).abs())), "lse")
    assert torch.equal(lse, moe.distill(z, ids, t)[1])
