"""distill, its gradient and the step in one call against the plain 64-bit form."""
import pytest
import torch

import _step_ref as ref
import top_routed_grouped_gb300 as moe

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def make(T, V, K, dtype, seed=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed * 99991 + T * 31 + V + K)
    z = (spread * torch.randn(T, V, generator=g, device="cuda")).to(dtype)
    part = V // K
    if part:
        ids = torch.arange(K, device="cuda") * part + torch.randint(part, (T, K), generator=g, device="cuda")
        ids = ids.gather(1, torch.rand(T, K, generator=g, device="cuda").argsort(1))
    else:
        ids = torch.randint(V, (T, K), generator=g, device="cuda")
    t = 2 * torch.randn(T, K, generator=g, device="cuda")
    return z, ids.int(), t, torch.randn(T, generator=g, device="cuda")


def all_ok(z, ids, t, w, tau=1.0, scale=1.0, t_lse=None, sums=None):
    """The three calls on one case; ``sums``: terms of a sum (the vocabulary's
    by default over the 128 threads or more that share a row)."""
    want = ref.distill(z, ids, t, tau, scale, t_lse, w)
    ops = ref.ROW + (z.shape[1] // 128 if sums is None else sums)
    loss, lse = moe.distill(z, ids, t, tau, scale, t_lse)
    ref.check(loss, *want["loss"], ops=ops, what="loss")
    ref.check(lse, *want["lse"], ops=ops, what="lse")
    d = moe.distill_backward(w, lse, z, ids, t, tau, scale, t_lse)
    assert d.dtype == z.dtype
    ref.check(d, *want["dlogits"], ops=ops, what="dlogits")
    loss2, d2 = moe.distill_step(z, ids, t, w, tau, scale, t_lse)
    ref.check(loss2, *want["loss"], ops=ops, what="loss of the step")
    ref.check(d2, *want["dlogits"], ops=ops, what="dlogits of the step")
    inplace = z.clone()
    loss3, d3 = moe.distill_step(inplace, ids, t, w, tau, scale, t_lse, out=inplace)
    assert d3 is inplace and torch.equal(d3.nan_to_num(7.0), d2.nan_to_num(7.0))
    assert torch.equal(loss3.nan_to_num(7.0), loss2.nan_to_num(7.0))
    inplace = z.clone()
    moe.distill_backward(w, lse, inplace, ids, t, tau, scale, t_lse, out=inplace)
    assert torch.equal(inplace.nan_to_num(7.0), d.nan_to_num(7.0))
    return loss, lse, d


@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (3, 2, 1), (5, 3, 3), (4, 17, 5), (2, 257, 256), (9, 1000, 8), (1, 4096, 64),
                                   (33, 5003, 33), (40, 32000, 20), (7, 50257, 200), (2, 262144, 256), (3, 300001, 7),
                                   (2, 1048576, 16)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_loss_and_gradient(T, V, K, dtype):
    all_ok(*make(T, V, K, dtype))


@pytest.mark.parametrize("tau,scale", [(2.0, 4.0), (0.5, -1.0), (7.3, 1.0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_temperature_and_scale(tau, scale, dtype):
    all_ok(*make(13, 3001, 12, dtype), tau=tau, scale=scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_teacher_with_its_own_normaliser(dtype):
    z, ids, t, w = make(20, 2000, 9, dtype)
    lse = torch.logsumexp(t, 1) + torch.rand(20, device="cuda")
    all_ok(z, ids, t, w, t_lse=lse)


@pytest.mark.parametrize("V", [100, 1003, 40000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slots_that_are_not_there(V, dtype):
    z, ids, t, w = make(24, V, 16, dtype)
    keep = torch.arange(24, device="cuda")[:, None] % 17
    ids = torch.where(torch.arange(16, device="cuda") < keep, ids, -1)  # row 0 and 17: none
    t[5, :3] = -INF
    t[6] = -INF  # none either
    t[7, 1:] = torch.finfo(F32).min
    w[3] = 0
    z[17] = float("nan")  # without slots its logits do not matter to the gradient
    z[3, 50] = float("nan")
    loss, lse = moe.distill(z, ids, t)
    d = moe.distill_backward(w, lse, z, ids, t)
    loss2, d2 = moe.distill_step(z, ids, t, w)
    want = ref.distill(z, ids, t, weight=w)
    for r in (0, 17, 6, 3):
        assert not d[r].any() and not d2[r].any(), r
    for r in (0, 17, 6):
        assert loss[r] == 0 and loss2[r] == 0, r
    rows = [r for r in range(24) if r not in (3, 17)]
    for got, name in ((loss, "loss"), (loss2, "loss"), (d, "dlogits"), (d2, "dlogits"), (lse, "lse")):
        v, m = want[name]
        ref.check(got[rows], v[rows], m[rows], ops=ref.ROW + V // 128, what=name)


@pytest.mark.parametrize("low", [-INF, torch.finfo(BF16).min])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [64, 5001])
def test_masked_vocabulary(low, dtype, V):
    """Student logits at -inf or at the type's lowest value; a teacher token
    among them; rows where one place is left, and none."""
    z, ids, t, w = make(6, V, 4, dtype)
    z[:, ::2] = low
    z[1, :] = low
    z[1, ids[1, 0].item()] = 1.5
    z[2, :] = -INF
    z[3, ids[3, 1].item()] = low
    ids[4] = 1  # only an open place, four times
    z[4, 1] = 0.0
    loss, lse = moe.distill(z, ids, t)
    d = moe.distill_backward(w, lse, z, ids, t)
    loss2, d2 = moe.distill_step(z, ids, t, w)
    want = ref.distill(z, ids, t, weight=w)
    assert loss[2] == INF and loss2[2] == INF and lse[2] == -INF and not d[2].any() and not d2[2].any()
    for got, name in ((loss, "loss"), (loss2, "loss"), (d, "dlogits"), (d2, "dlogits"), (lse, "lse")):
        v, m = want[name]
        if name != "dlogits":
            got = got.clone()
        ref.check(got, v, m, ops=ref.ROW + V // 128, what=name)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nan_and_inf_stay_in_their_rows(dtype):
    z, ids, t, w = make(5, 3000, 6, dtype)
    z[1, 2999] = float("nan")
    z[3, 10] = INF
    loss, lse = moe.distill(z, ids, t)
    loss2, d2 = moe.distill_step(z, ids, t, w)
    d = moe.distill_backward(w, lse, z, ids, t)
    for x in (loss, loss2, lse):
        assert torch.isnan(x[[1, 3]]).all() and torch.isfinite(x[[0, 2, 4]]).all()
    for x in (d, d2):
        assert torch.isnan(x[[1, 3]]).all() and torch.isfinite(x[[0, 2, 4]]).all()


def test_duplicates_and_bad_ids():
    z, ids, t, w = make(8, 700, 10, F32)
    ids[:, 3] = ids[:, 0]
    ids[:, 7] = ids[:, 0]
    moe.moe_device_status(reset=True)
    all_ok(z, ids, t, w)
    assert moe.moe_device_status(reset=True) == 0
    ids[2, 4], ids[5, 1] = 700, -2
    loss, d = moe.distill_step(z, ids, t, w)
    assert moe.moe_device_status(reset=True) == 6
    want = ref.distill(z, ids, t, weight=w)
    ref.check(loss, *want["loss"], ops=ref.ROW + 8, what="loss")
    ref.check(d, *want["dlogits"], ops=ref.ROW + 8, what="dlogits")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,shift,pad", [(1000, 0, 24), (1001, 1, 0), (999, 3, 5), (40007, 5, 1)])
def test_strided_rows(dtype, V, shift, pad):
    z, ids, t, w = make(11, V, 8, dtype)
    wide = torch.full((11, V + shift + pad), float("nan"), device="cuda", dtype=dtype)
    wide[:, shift:shift + V] = z
    view = wide[:, shift:shift + V]
    want = ref.distill(z, ids, t, weight=w)
    loss, d = moe.distill_step(view, ids, t, w, out=view)
    ref.check(loss, *want["loss"], ops=ref.ROW + V // 128, what="loss")
    ref.check(d, *want["dlogits"], ops=ref.ROW + V // 128, what="dlogits")
    assert torch.isnan(wide[:, :shift]).all() and torch.isnan(wide[:, shift + V:]).all()  # nothing beside the rows


@pytest.mark.parametrize("dtype,V", [(F32, 5003), (BF16, 32000), (BF16, 50257), (BF16, 131072)])
def test_rows_do_not_depend_on_the_batch(dtype, V):
    """Within one launch shape a row's bits are its own; across batch sizes
    (few rows are split over more of the GPU) they agree to rounding."""
    z, ids, t, w = make(400, V, 8, dtype)
    full = moe.distill_step(z, ids, t, w)
    again = moe.distill_step(z, ids, t, w)
    assert torch.equal(full[0], again[0]) and torch.equal(full[1], again[1])
    perm = torch.randperm(400, device="cuda")
    moved = moe.distill_step(z[perm], ids[perm], t[perm], w[perm])
    assert torch.equal(moved[0], full[0][perm]) and torch.equal(moved[1], full[1][perm])
    want = ref.distill(z[3:5], ids[3:5], t[3:5], weight=w[3:5])
    few = moe.distill_step(z[3:5], ids[3:5], t[3:5], w[3:5])
    ref.check(few[0], *want["loss"], ops=ref.ROW + V // 128, what="loss")
    ref.check(few[1], *want["dlogits"], ops=ref.ROW + V // 128, what="dlogits")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,ld", [(900, 901), (5003, 5003), (16384, 16385), (32000, 32003), (32000, 32008), (131072, 131073)])
def test_rows_are_the_same_bits_in_any_batch(dtype, V, ld):
    """The shape goes by the vocabulary and the rows' alignment alone: any rows
    of a batch, one of them too, have the bits that they have in the whole."""
    z, ids, t, w = make(150, V, 8, dtype)
    rows = torch.zeros(149 * ld + V, device="cuda", dtype=dtype).as_strided((150, V), (ld, 1))
    rows.copy_(z)
    loss, lse = moe.distill(rows, ids, t)
    step = moe.distill_step(rows, ids, t, w)
    d = moe.distill_backward(w, lse, rows, ids, t)
    for i in (slice(0, 1), slice(3, 5), slice(8, 9), slice(149, 150), slice(20, 111)):
        p = moe.distill(rows[i], ids[i], t[i])
        assert torch.equal(p[0], loss[i]) and torch.equal(p[1], lse[i])
        p = moe.distill_step(rows[i], ids[i], t[i], w[i])
        assert torch.equal(p[0], step[0][i]) and torch.equal(p[1], step[1][i])
        assert torch.equal(moe.distill_backward(w[i], lse[i], rows[i], ids[i], t[i]), d[i])


def test_rows_past_32_bit_offsets():
    T, V = 20000, 131072  # 2.6e9 elements
    z = torch.zeros(T, V, dtype=BF16, device="cuda")
    ids = torch.full((T, 1), V - 1, dtype=torch.int32, device="cuda")
    t = torch.zeros(T, 1, device="cuda")
    z[T - 1, V - 1] = 4.0
    loss, d = moe.distill_step(z, ids, t, torch.ones(T, device="cuda"), out=z)
    n = torch.log(torch.tensor(float(V), dtype=torch.float64))
    last = torch.log(torch.exp(torch.tensor(4.0, dtype=torch.float64)) + V - 1) - 4
    assert abs(float(loss[0]) - float(n)) < 1e-4 and abs(float(loss[-1]) - float(last)) < 1e-4
    assert float(d[T - 1, V - 1]) == pytest.approx(float(torch.exp(-last)) - 1, rel=2 ** -8)
    assert float(d[T - 2, V - 1]) == pytest.approx(1 / V - 1, rel=2 ** -8)
    assert float(d[T - 1, 5]) == pytest.approx(float(torch.exp(-last - 4)), rel=2 ** -8)


def test_gradient_against_differences():
    """Central differences of sum(w loss) along random directions.  Cut-off
    error of step 1e-2 and the losses' roundings (2^-24 of about 20, over the
    step) are below 1e-3 of the derivative's terms."""
    z, ids, t, w = make(6, 500, 5, F32, spread=1.0)
    w = w.abs() + 0.5
    for tau, t_lse in ((1.0, None), (2.0, torch.logsumexp(t / 2.0, 1) + 0.3)):
        f = lambda x: float((moe.distill(x, ids, t, tau, 1.5, t_lse)[0].double() * w.double()).sum())  # noqa: E731
        grad = moe.distill_step(z, ids, t, w, tau, 1.5, t_lse)[1]
        g = torch.Generator(device="cuda").manual_seed(1)
        v = torch.randn(z.shape, generator=g, device="cuda")
        num = (f(z + 1e-2 * v) - f(z - 1e-2 * v)) / 2e-2
        terms = grad.double() * v.double()
        assert abs(num - float(terms.sum())) <= 2e-3 * float(terms.abs().sum())


def test_side_stream_and_no_rows():
    z, ids, t, w = make(30, 8192, 8, BF16)
    want = moe.distill_step(z, ids, t, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.distill_step(z, ids, t, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    loss, d = moe.distill_step(z[:0], ids[:0], t[:0], w[:0])
    assert loss.shape == (0,) and d.shape == (0, 8192)


def test_refusals():
    z, ids, t, w = make(4, 64, 3, F32)
    for f in (lambda: moe.distill(z.half(), ids, t), lambda: moe.distill(z, ids.long(), t),
              lambda: moe.distill(z, ids[:3], t), lambda: moe.distill(z, ids, t.to(BF16)),
              lambda: moe.distill(z.cpu(), ids, t), lambda: moe.distill(z, ids, t, t_lse=w[:2]),
              lambda: moe.distill_step(z, ids, t, w[:3]), lambda: moe.distill_step(z, ids, t, w, out=z.to(BF16)),
              lambda: moe.distill_step(z, ids, t, w, out=torch.empty(64, 4, device="cuda").t())):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: moe.distill(z, ids, t, temperature=0.0), lambda: moe.distill(z, ids, t, temperature=-1.0),
              lambda: moe.distill(z, ids, t, scale=float("nan")),
              lambda: moe.distill(z, torch.zeros(4, 257, dtype=torch.int32, device="cuda"), torch.zeros(4, 257, device="cuda"))):
        with pytest.raises(moe.MoEError):
            f()
