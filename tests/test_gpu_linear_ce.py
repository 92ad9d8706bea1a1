"""linear_cross_entropy, its gradient and step against plain forms in 64 bits."""
import ctypes

import pytest
import torch

import top_routed_grouped_gb300 as moe
from _train_ref import IGNORE, check, cross_entropy

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16


def status():
    detail = ctypes.c_int32(0)
    rc = moe.lib().moe_device_status(1, ctypes.byref(detail))
    return detail.value if rc else 0


def make(T, D, V, dtype, seed=0, left_out=0, spread=2.0, ids=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = rn(V, D) * (spread / D ** 0.5)
    t = torch.randint(V, (T,), generator=g, device="cuda")
    h = rn(T, D) + torch.rand(T, 1, generator=g, device="cuda") * 1.5 * w[t]
    if left_out:
        t[torch.randperm(T, generator=g, device="cuda")[:left_out]] = IGNORE
    d = (0.5 + torch.rand(T, generator=g, device="cuda")) / max(T, 1)
    return h.to(dtype), w.to(dtype), t.to(ids), d


def all_ok(h, w, t, d, scale=1.0, z=0.0):
    kw = dict(scale=scale, z_loss=z)
    ref = cross_entropy(h, w, t, d, scale, z)
    loss, lse = moe.linear_cross_entropy(h, w, t, **kw)
    check(loss, ref["loss"], "loss")
    check(lse, ref["lse"], "lse")
    dh, dw = moe.linear_cross_entropy_backward(d, lse, h, w, t, **kw)
    assert dh.dtype is h.dtype and dw.dtype is w.dtype
    check(dh, ref["dhidden"], "dhidden")
    check(dw, ref["dweight"], "dweight")
    loss2, dh2, dw2 = moe.linear_cross_entropy_step(h, w, t, d, **kw)
    assert torch.equal(loss2, loss)
    check(dh2, ref["dhidden"], "dhidden of the step")
    check(dw2, ref["dweight"], "dweight of the step")
    assert status() == 0


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("T,D,V", [(1, 1, 1), (1, 64, 1000), (1, 77, 65), (2, 8, 63), (3, 130, 64), (31, 128, 129),
                                   (33, 64, 257), (65, 256, 255), (128, 63, 2000), (255, 72, 300), (257, 520, 513),
                                   (300, 100, 1111), (700, 256, 8193)])
def test_sizes(T, D, V, dtype):
    all_ok(*make(T, D, V, dtype))


@pytest.mark.parametrize("T,D,V", [(4097, 64, 20000), (5600, 136, 17000), (130, 1032, 40000), (2049, 1000, 9000),
                                   (20011, 72, 8300)])
def test_larger_sizes(T, D, V):
    all_ok(*make(T, D, V, B, left_out=T // 3))


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("scale,z", [(0.25, 0.0), (-1.0, 1e-3), (4.0, 1e-4), (0.0, 0.0), (1.0, 0.5)])
def test_scale_and_z_loss(scale, z, dtype):
    all_ok(*make(140, 96, 700, dtype, left_out=20), scale=scale, z=z)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("T,left_out", [(1, 1), (64, 64), (64, 63), (300, 1), (513, 257), (5000, 4990), (4500, 4500)])
def test_rows_that_are_left_out_are_not_read(T, left_out, dtype):
    """Whatever such rows hold; their loss, lse and dhidden are 0, dweight has nothing of them."""
    h, w, t, d = make(T, 72, 333, dtype, left_out=left_out)
    out = t == IGNORE
    h[out] = torch.tensor(float("nan"), device="cuda", dtype=dtype)
    h[out.nonzero()[::2, 0]] = torch.tensor(float("inf"), device="cuda", dtype=dtype)
    d[out] = float("nan")
    all_ok(h, w, t, d)
    loss, lse = moe.linear_cross_entropy(h, w, t)
    loss2, dh, _ = moe.linear_cross_entropy_step(h, w, t, d)
    for v in (loss, lse, loss2, dh):
        assert not v[out].any()


def test_targets_outside_the_vocabulary():
    h, w, t, d = make(40, 64, 100, B)
    bad = t.clone()
    bad[3], bad[7] = 100, -7
    want = t.clone()
    want[3] = want[7] = IGNORE
    for f in (lambda i: moe.linear_cross_entropy(h, w, i), lambda i: moe.linear_cross_entropy_step(h, w, i, d)):
        got = f(bad)
        assert status() == 7
        assert all(torch.equal(a, b) for a, b in zip(got, f(want)))
        assert status() == 0
    # Another value to ignore; -100 is outside then.
    again = moe.linear_cross_entropy(h, w, torch.where(want == IGNORE, 5, want).int(), ignore_index=5)[0]
    five = want == 5
    ref = moe.linear_cross_entropy(h, w, want)[0]
    assert status() == 0 and torch.equal(again[~five], ref[~five]) and not again[five].any()
    moe.linear_cross_entropy(h, w, want, ignore_index=5)
    assert status() == 7


@pytest.mark.parametrize("dtype", [F, B])
def test_targets_of_32_bits(dtype):
    h, w, t, d = make(77, 64, 130, dtype, left_out=9)
    for a, b in zip(moe.linear_cross_entropy_step(h, w, t, d), moe.linear_cross_entropy_step(h, w, t.int(), d)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (3, 5), (8, 1)])
def test_strides_and_alignment(shift, pad, dtype):
    """Rows between others' bytes and off the 16-byte boundaries: the values of dense ones."""
    T, D, V = 90, 104, 401
    h, w, t, d = make(T, D, V, dtype, left_out=11)

    def within(x):
        rows = torch.full((x.shape[0], D + pad + shift), float("nan"), device="cuda", dtype=dtype)
        view = rows[:, shift:shift + D]
        view.copy_(x)
        return view

    want = moe.linear_cross_entropy_step(h, w, t, d)
    for hh, ww in ((within(h), w), (h, within(w)), (within(h), within(w))):
        for a, b in zip(moe.linear_cross_entropy_step(hh, ww, t, d), want):
            assert torch.equal(a, b)
    for a, b in zip(moe.linear_cross_entropy_step(h.t().contiguous().t(), w.t().contiguous().t(), t, d), want):
        assert torch.equal(a, b)
    one = h[:1].expand(T, D)
    for a, b in zip(moe.linear_cross_entropy_step(one, w, t, d), moe.linear_cross_entropy_step(one.contiguous(), w, t, d)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 100, 77])
def test_dweight_in_float32_and_added_to(D):
    h, w, t, d = make(150, D, 301, B, left_out=10)
    ref = cross_entropy(h, w, t, d)
    _, lse = moe.linear_cross_entropy(h, w, t)
    dh, dw = moe.linear_cross_entropy_backward(d, lse, h, w, t, dweight_dtype=F)
    assert dw.dtype is F
    check(dw, ref["dweight32"], "dweight in float32")
    plain = moe.linear_cross_entropy_backward(d, lse, h, w, t)[1]
    assert torch.equal(plain, dw.bfloat16())
    base = torch.randn(301, D, device="cuda")
    acc = base.clone()
    version = acc._version
    assert moe.linear_cross_entropy_backward(d, lse, h, w, t, dweight=acc)[1] is acc
    assert acc._version > version and torch.equal(acc, base + dw)
    hf, wf = h.float(), w.float()
    _, dhf, dwf = moe.linear_cross_entropy_step(hf, wf, t, d)
    acc = base.clone()
    moe.linear_cross_entropy_step(hf, wf, t, d, dweight=acc)
    assert torch.equal(acc, base + dwf)
    nothing = torch.full_like(t, IGNORE)  # no row at all: zeros, or what was there
    assert not moe.linear_cross_entropy_step(h, w, nothing, d)[2].any()
    acc = base.clone()
    moe.linear_cross_entropy_step(h, w, nothing, d, dweight=acc)
    assert torch.equal(acc, base)


@pytest.mark.parametrize("dtype,T,D,V", [(B, 6000, 64, 20000), (B, 700, 200, 33000), (F, 900, 40, 1700)])
def test_rows_are_the_same_bits_in_any_batch(dtype, T, D, V):
    """Alone, among others, and with others left out; pieces and planes differ with the batch."""
    h, w, t, d = make(T, D, V, dtype)
    loss, lse = moe.linear_cross_entropy(h, w, t)
    dh, _ = moe.linear_cross_entropy_backward(d, lse, h, w, t)
    _, dh_step, _ = moe.linear_cross_entropy_step(h, w, t, d)
    for a, b in ((0, 1), (5, 70), (T - 300, T)):
        s = slice(a, b)
        l2, e2 = moe.linear_cross_entropy(h[s], w, t[s])
        assert torch.equal(l2, loss[s]) and torch.equal(e2, lse[s])
        assert torch.equal(moe.linear_cross_entropy_backward(d[s], e2, h[s], w, t[s])[0], dh[s])
        assert torch.equal(moe.linear_cross_entropy_step(h[s], w, t[s], d[s])[1], dh_step[s])
    some = t.clone()
    some[::3] = IGNORE
    keep = some != IGNORE
    l3, dh3, _ = moe.linear_cross_entropy_step(h, w, some, d)
    assert torch.equal(l3[keep], loss[keep]) and torch.equal(dh3[keep], dh_step[keep])


@pytest.mark.parametrize("dtype", [F, B])
def test_the_same_bits_every_time(dtype):
    h, w, t, d = make(400, 200, 9000, dtype, left_out=50)
    first = moe.linear_cross_entropy_step(h, w, t, d)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(moe.linear_cross_entropy_step(h, w, t, d), first))


@pytest.mark.parametrize("dtype", [F, B])
def test_sure_rows(dtype):
    """Targets far above the others: the loss is small, not lost in lse; and far below."""
    T, D, V = 64, 64, 500
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(V, D, generator=g, device="cuda") * 0.05
    t = torch.arange(T, device="cuda") * 7 % V
    w[t, torch.arange(T, device="cuda")] += 1.0
    h = torch.zeros(T, D, device="cuda")
    h[torch.arange(T), torch.arange(T)] = torch.linspace(-60, 60, T, device="cuda")
    all_ok(h.to(dtype), w.to(dtype), t, torch.rand(T, generator=g, device="cuda"))


def test_infinities_and_nan_stay_in_their_rows():
    h, w, t, d = make(70, 64, 400, B)
    want = moe.linear_cross_entropy_step(h, w, t, d)
    hh = h.clone()
    hh[3, 5], hh[40, 0] = float("nan"), float("inf")
    loss, dh, _ = moe.linear_cross_entropy_step(hh, w, t, d)
    rest = torch.ones(70, dtype=torch.bool, device="cuda")
    rest[[3, 40]] = False
    assert not torch.isfinite(loss[~rest]).any()
    assert torch.equal(loss[rest], want[0][rest]) and torch.equal(dh[rest], want[1][rest])
    assert not torch.isfinite(dh[~rest]).all(1).any()


@pytest.mark.parametrize("dtype,D,pad,shift", [(B, 64, 16, 0), (B, 64, 8, 1), (B, 77, 3, 2), (F, 60, 4, 1)])
def test_dhidden_between_others_bytes(dtype, D, pad, shift):
    """Through the C entry points: rows with a stride, off any wide boundary; what lies between them stays."""
    from top_routed_grouped_gb300 import train
    T, V = 70, 300
    h, w, t, d = make(T, D, V, dtype, left_out=9)
    _, lse = moe.linear_cross_entropy(h, w, t)
    want = moe.linear_cross_entropy_backward(d, lse, h, w, t)
    rows = torch.full((T * (D + pad) + shift,), 5.0, device="cuda", dtype=dtype)
    dw = torch.empty_like(w)
    code = 0 if dtype is F else 1
    args = train._CE.pack(T, D, V, code, code, 0, 1, 1.0, 0.0, 0, -100, 0, 0, D + pad, h.data_ptr(), w.data_ptr(),
                          t.data_ptr(), d.data_ptr(), 0, lse.data_ptr(), rows.data_ptr() + shift * rows.element_size(),
                          dw.data_ptr())
    n = train.moe_linear_ce_workspace_size(args, 2)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    train.moe_linear_ce_backward(args, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    view = rows[shift:].view(T, D + pad)
    assert torch.equal(view[:, :D], want[0]) and torch.equal(dw, want[1])
    assert bool((view[:, D:] == 5).all()) and bool((rows[:shift] == 5).all())


@pytest.mark.parametrize("D", [64, 72, 77])
def test_dweight_off_any_boundary(D):
    """A gradient that starts between 16-byte boundaries takes another path to memory."""
    from top_routed_grouped_gb300 import train
    T, V = 70, 300
    h, w, t, d = make(T, D, V, B)
    for dtype, accumulate in ((B, 0), (F, 0), (F, 1)):
        flat = torch.full((V * D + 6,), 5.0, device="cuda", dtype=dtype)
        want = moe.linear_cross_entropy_step(h, w, t, d, dweight_dtype=dtype)[2]
        dh, loss = torch.empty_like(h), torch.empty(T, device="cuda")
        args = train._CE.pack(T, D, V, 1, 0 if dtype is F else 1, accumulate, 1, 1.0, 0.0, 0, -100, 0, 0, 0, h.data_ptr(),
                              w.data_ptr(), t.data_ptr(), d.data_ptr(), loss.data_ptr(), 0, dh.data_ptr(),
                              flat.data_ptr() + 3 * flat.element_size())
        n = train.moe_linear_ce_workspace_size(args, 3)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        train.moe_linear_ce_step(args, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        assert torch.equal(flat[3:-3].view(V, D), want + 5 if accumulate else want)
        assert bool((flat[:3] == 5).all()) and bool((flat[-3:] == 5).all())


def test_dloss_of_zero():
    h, w, t, d = make(70, 64, 400, B)
    d[10:20] = 0
    all_ok(h, w, t, d)
    assert not moe.linear_cross_entropy_step(h, w, t, d)[1][10:20].any()


def test_gradient_against_differences():
    """In float32: (L(h + e) - L(h - e)) / 2 against dhidden . e, and the weights'
    alike.  With steps of 2^-5 the third derivative leaves about 2^-10 / 6 of the
    size of e cubed (here a unit vector over logits of slope 1: below 2e-4), and
    the losses' roundings (32 rows' loss of 2^-20 over 2^-4): 1e-4."""
    T, D, V = 32, 48, 90
    h, w, t, d = make(T, D, V, F, left_out=4)
    d = torch.rand(T, device="cuda") / T
    kw = dict(scale=0.7, z_loss=1e-2)
    total = lambda h, w: float((moe.linear_cross_entropy(h, w, t, **kw)[0].double() * d).sum())  # noqa: E731
    _, dh, dw = moe.linear_cross_entropy_step(h, w, t, d, **kw)
    g = torch.Generator(device="cuda").manual_seed(5)
    for _ in range(4):
        for x, grad, f in ((h, dh, lambda e: total(h + e, w) - total(h - e, w)),
                           (w, dw, lambda e: total(h, w + e) - total(h, w - e))):
            e = torch.randn(x.shape, generator=g, device="cuda")
            e *= 2.0 ** -5 / float(e.norm())
            assert abs(f(e) / 2 - float((grad * e).sum())) <= 2.0 ** -5 * 3e-4


def test_no_rows():
    w = torch.randn(50, 64, device="cuda").bfloat16()
    h, t, d = w[:0], torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = moe.linear_cross_entropy(h, w, t)
    assert loss.shape == lse.shape == (0,)
    loss, dh, dw = moe.linear_cross_entropy_step(h, w, t, d)
    assert dh.shape == (0, 64) and not dw.any() and dw.shape == w.shape
    acc = torch.ones(50, 64, device="cuda")
    moe.linear_cross_entropy_step(h, w, t, d, dweight=acc)
    assert bool((acc == 1).all())


def test_table_past_32_bit_offsets():
    """2^31 elements and more in the weights and in their gradient; a few targets at the end."""
    V, D = 1 << 20, 2056
    w = torch.empty(V, D, dtype=B, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for a in range(0, V, 1 << 16):
        w[a:a + (1 << 16)] = torch.randn(1 << 16, D, generator=g, device="cuda").mul_(1.5 / D ** 0.5)
    t = torch.tensor([V - 1, 0, V // 2 + 3, V - 1], device="cuda")
    h = (torch.randn(4, D, generator=g, device="cuda") + 2 * w[t].float()).to(B)
    d = torch.tensor([0.5, 1.0, 2.0, 0.25], device="cuda")
    loss, dh, dw = moe.linear_cross_entropy_step(h, w, t, d)
    rows = torch.cat([torch.arange(0, 300, device="cuda"), torch.arange(V - 300, V, device="cuda"), t[2:3]])
    x = torch.cat([h.double() @ w[a:a + (1 << 16)].double().t() for a in range(0, V, 1 << 16)], 1)
    lse = torch.logsumexp(x, 1)
    mag = max(float((h.double().abs() @ w[a:a + (1 << 16)].double().abs().t()).max()) for a in range(0, V, 1 << 16))
    tol = 3 * (D + 8) * 2.0 ** -23 * mag + (V / 64 + 80) * 2.0 ** -24  # (as in cross_entropy)
    assert float((loss - (lse - x.gather(1, t[:, None])[:, 0])).abs().max()) <= tol
    p = torch.exp(x - lse[:, None]) * d[:, None].double()
    p.scatter_add_(1, t[:, None], -d[:, None].double())
    want = torch.einsum("tv,td->vd", p[:, rows], h.double())
    mag = torch.einsum("tv,td->vd", p[:, rows].abs(), h.double().abs())
    # Three roundings to bfloat16; p by the same logits as the loss.
    assert bool(((dw[rows] - want).abs() <= (3 * 2.0 ** -8 + 2 * tol) * mag).all())
    dwant = sum(p[:, a:a + (1 << 16)] @ w[a:a + (1 << 16)].double() for a in range(0, V, 1 << 16))
    dmag = sum(p[:, a:a + (1 << 16)].abs() @ w[a:a + (1 << 16)].double().abs() for a in range(0, V, 1 << 16))
    assert bool(((dh - dwant).abs() <= (2 * 2.0 ** -8 + 2 * tol) * dmag).all())


def test_workspaces_and_streams():
    h, w, t, d = make(120, 64, 900, B, left_out=7)
    want = moe.linear_cross_entropy_step(h, w, t, d)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # what it holds does not matter
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in (dict(ws=ws), dict(stream=side), dict(ws=ws, stream=side.cuda_stream)):
        got = moe.linear_cross_entropy_step(h, w, t, d, **kw)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(moe.MoEError):
        moe.linear_cross_entropy_step(h, w, t, d, ws=ws[:1024])
    with pytest.raises(moe.MoEError):
        moe.linear_cross_entropy(h, w, t, ws=ws[16:])
    with pytest.raises(ValueError):
        moe.linear_cross_entropy(h, w, t, ws=ws.cpu())
    with pytest.raises(ValueError):
        moe.linear_cross_entropy(h, w, t, ws=ws[::2])


def test_calls_one_after_another_in_one_workspace():
    """Kernels start while those before them finish: calls of different sizes, types and numbers of
    rows, through one workspace and without a pause, see nothing of one another."""
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    cases = [make(T, D, V, dtype, seed=i, left_out=left) for i, (T, D, V, dtype, left) in enumerate(
        [(300, 200, 9000, B, 20), (5, 64, 100, F, 0), (5000, 64, 3000, B, 4000), (1, 8, 20000, B, 0), (700, 72, 500, F, 100),
         (64, 512, 17000, B, 63)])]
    want = [moe.linear_cross_entropy_step(*c) for c in cases]
    torch.cuda.synchronize()
    got = [moe.linear_cross_entropy_step(*cases[i], ws=ws) for _ in range(6) for i in range(6)]
    losses = [moe.linear_cross_entropy(*cases[i % 6][:3], ws=ws)[0] for i in range(30)]
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 6])), i
    for i, loss in enumerate(losses):
        assert torch.equal(loss, want[i % 6][0]), i
    assert status() == 0


@pytest.mark.parametrize("dtype", [F, B])
def test_captured_and_replayed(dtype):
    """Other rows, other targets, another number of rows that count."""
    T, D, V = 200, 72, 1500
    h, w, t, d = make(T, D, V, dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.linear_cross_entropy_step(h, w, t, d)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = moe.linear_cross_entropy_step(h, w, t, d)
    for seed, left_out in ((1, 0), (2, 150), (3, 200), (4, 5)):
        h2, w2, t2, d2 = make(T, D, V, dtype, seed=seed, left_out=left_out)
        for a, b in ((h, h2), (w, w2), (t, t2), (d, d2)):
            a.copy_(b)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, moe.linear_cross_entropy_step(h2, w2, t2, d2)))


def test_refusals():
    h, w, t, d = make(20, 64, 90, B)
    loss, lse = moe.linear_cross_entropy(h, w, t)
    bad = [
        lambda: moe.linear_cross_entropy(h.float(), w, t),
        lambda: moe.linear_cross_entropy(h.half(), w.half(), t),
        lambda: moe.linear_cross_entropy(h[:, :32], w, t),
        lambda: moe.linear_cross_entropy(h[None], w, t),
        lambda: moe.linear_cross_entropy(h, w[0], t),
        lambda: moe.linear_cross_entropy(h, w, t[:10]),
        lambda: moe.linear_cross_entropy(h, w, t.float()),
        lambda: moe.linear_cross_entropy(h, w, t[:, None]),
        lambda: moe.linear_cross_entropy(h, w, t.cpu()),
        lambda: moe.linear_cross_entropy(h, w.cpu(), t),
        lambda: moe.linear_cross_entropy(h.cpu(), w, t),
        lambda: moe.linear_cross_entropy_step(h, w, t, d.double()),
        lambda: moe.linear_cross_entropy_step(h, w, t, d[:5]),
        lambda: moe.linear_cross_entropy_step(h, w, t, d, dweight=torch.zeros_like(w)),
        lambda: moe.linear_cross_entropy_step(h, w, t, d, dweight=torch.zeros(90, 32, device="cuda")),
        lambda: moe.linear_cross_entropy_step(h, w, t, d, dweight=torch.zeros(64, 90, device="cuda").t()),
        lambda: moe.linear_cross_entropy_step(h, w, t, d, dweight_dtype=torch.float16),
        lambda: moe.linear_cross_entropy_backward(d, lse[:3], h, w, t),
        lambda: moe.linear_cross_entropy_backward(d, lse.double(), h, w, t),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for kw in (dict(scale=float("nan")), dict(z_loss=-1.0), dict(z_loss=float("inf"))):
        with pytest.raises(moe.MoEError):
            moe.linear_cross_entropy(h, w, t, **kw)
    assert status() == 0
