"""block_norm and its gradients against the plain 64-bit form."""
import pytest
import torch

import _step_ref as ref
import top_routed_grouped_gb300 as moe

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6
INF = float("inf")


def make(T, H, dtype, rdtype, wdtype, post=True, pre=True, block=True, gate="none", offset=0.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + 7 * T + H)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    c = {"r": rn(T, H).to(rdtype), "y": rn(T, H).to(dtype) if block else None,
         "w_post": (1 - offset + 0.2 * rn(H)).to(wdtype) if post and block else None,
         "w_pre": (1 - offset + 0.2 * rn(H)).to(wdtype) if pre else None, "gate": None}
    if block:
        c["gate"] = {"none": lambda: None, "token": lambda: rn(T, 1), "channel": lambda: rn(H).to(wdtype),
                     "element": lambda: rn(T, H).to(dtype)}[gate]()
    c["dr_out"], c["dh"] = rn(T, H).to(rdtype), rn(T, H).to(dtype) if pre else None
    return c


def forward_ok(c, dtype, scale, offset, **kw):
    r_out, h = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"], scale=scale, eps=EPS,
                              weight_offset=offset, dtype=dtype, **kw)
    want = ref.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"], scale, EPS, offset)
    if c["y"] is not None:
        assert r_out.dtype == c["r"].dtype
        ref.check(r_out, *want["r_out"], what="r_out")
    else:
        assert r_out is c["r"]
    if c["w_pre"] is not None:
        assert h.dtype == dtype
        ref.check(h, *want["h"], what="h")
    else:
        assert h is None
    return r_out, h


def backward_ok(c, r_out, scale, offset):
    got = moe.block_norm_backward(c["dr_out"], c["dh"], r_out, c["y"], c["w_post"], c["w_pre"], c["gate"],
                                  scale=scale, eps=EPS, weight_offset=offset)
    want = ref.block_norm_backward(c["dr_out"], c["dh"], r_out, c["y"], c["w_post"], c["w_pre"], c["gate"], scale,
                                   EPS, offset)
    T = c["r"].shape[0]
    for name in ("dr", "dy", "dw_post", "dw_pre", "dgate"):
        assert (got[name] is None) == (name not in want), name
        if name in want:
            sums = name.startswith("dw") or (name == "dgate" and c["gate"].dim() == 1)
            tokens = name == "dgate" and c["gate"].dim() == 2 and c["gate"].shape[1] == 1
            ref.check(got[name], *want[name], ops=ref.ROW + (T if sums else 0) + (64 if tokens else 0), what=name)
    return got


TYPES = [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, F32), (BF16, F32, BF16), (BF16, BF16, F32)]


@pytest.mark.parametrize("T,H", [(1, 1), (3, 2), (5, 7), (2, 31), (33, 64), (9, 100), (4, 257), (37, 256), (1, 2048),
                                 (700, 1001), (513, 2048), (6, 4104), (3, 8192), (2, 11111), (2, 16384)])
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x).split(".")[1] for x in t))
def test_join_and_gradients(T, H, types):
    c = make(T, H, *types, gate="none")
    r_out, _ = forward_ok(c, types[0], 0.5, 0.0)
    backward_ok(c, r_out, 0.5, 0.0)


@pytest.mark.parametrize("gate", ["none", "token", "channel", "element"])
@pytest.mark.parametrize("post,pre,block", [(True, True, True), (False, True, True), (True, False, True),
                                            (False, False, True), (False, True, False)])
@pytest.mark.parametrize("T,H", [(35, 96), (12, 77), (130, 2048)])
@pytest.mark.parametrize("types", TYPES[:3], ids=lambda t: "-".join(str(x).split(".")[1] for x in t))
def test_forms(gate, post, pre, block, T, H, types):
    if not block and gate != "none":
        pytest.skip("a gate belongs to y")
    c = make(T, H, *types, post=post, pre=pre, block=block, gate=gate, offset=1.0)
    r_out, _ = forward_ok(c, types[0], -1.5, 1.0)
    if block or pre:
        backward_ok(c, r_out, -1.5, 1.0)


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x).split(".")[1] for x in t))
def test_token_gate_of_one_channel(types):
    """A float gate [T, 1] is a token's where rows have one channel, too."""
    c = make(70, 1, *types, gate="token")
    r_out, _ = forward_ok(c, types[0], 0.5, 0.0)
    backward_ok(c, r_out, 0.5, 0.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_upstream_for_the_residual(dtype):
    c = make(19, 320, dtype, F32, F32, gate="element")
    c["dr_out"] = None
    r_out, _ = forward_ok(c, dtype, 1.0, 0.0)
    backward_ok(c, r_out, 1.0, 0.0)


@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 3), (8, 24), (3, 0)])
@pytest.mark.parametrize("types", TYPES[:3], ids=lambda t: "-".join(str(x).split(".")[1] for x in t))
def test_strided_and_misaligned_rows(shift, pad, types):
    """Rows that are windows of wider ones, each tensor at its own offset."""
    c = make(21, 264, *types, gate="element")

    def window(t, s):
        wide = torch.full((t.shape[0], t.shape[1] + shift + pad + s), float("nan"), device="cuda", dtype=t.dtype)
        wide[:, s + shift:s + shift + t.shape[1]] = t
        return wide[:, s + shift:s + shift + t.shape[1]]

    dense = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"])
    w = dict(c, **{n: window(c[n], 8 * i) for i, n in enumerate(("r", "y", "gate", "dr_out", "dh"))})
    r_out, h = forward_ok(w, types[0], 1.0, 0.0)
    if (264 + shift + pad) % 8 == 0 and shift % 8 == 0:
        assert torch.equal(r_out, dense[0]) and torch.equal(h, dense[1])
    backward_ok(w, window(r_out, 0), 1.0, 0.0)


def windows(c, ld, at):
    """The rows of ``c`` as windows of buffers of NaN: row stride ``ld``, from
    element ``at`` on, each tensor's buffer ending with its last row."""
    def window(t):
        T, H = t.shape
        buf = torch.full((at + (T - 1) * ld + H,), float("nan"), device="cuda", dtype=t.dtype)
        w = buf.as_strided((T, H), (ld, 1), at)
        w.copy_(t)
        return w

    return dict(c, **{n: window(c[n]) for n in ("r", "y", "gate", "dr_out", "dh")}), window


@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 6, 7, 9, 12])
@pytest.mark.parametrize("types", TYPES[:3], ids=lambda t: "-".join(str(x).split(".")[1] for x in t))
def test_narrow_rows_at_any_place(types, H):
    """Rows of a few bytes: several lie in the first and in the last 16 bytes of
    their buffer, dense at every offset from a 16-byte boundary or strided."""
    for T in (3, 5, 10, 12, 65, 66, 129, 130, 193):
        c = make(T, H, *types, gate="element", seed=T)
        for ld, at in [(H, n) for n in range(8)] + [(H + 1, 0), (H + 1, 1), (H + 2, 3), (H + 5, 0), (H + 5, 7)]:
            w, window = windows(c, ld, at)
            r_out, _ = forward_ok(w, types[0], 1.0, 0.0)
            backward_ok(w, window(r_out), 1.0, 0.0)


@pytest.mark.parametrize("types,T,H", [(TYPES[0], 9001, 333), (TYPES[1], 9001, 1001), (TYPES[2], 40001, 77)])
def test_long_walks_from_a_misaligned_start(types, T, H):
    """The stage of the first block, whose start is filled in by hand, is
    copied to many times after it."""
    c = make(T, H, *types, gate="element")
    w, window = windows(c, H, 1)
    r_out, _ = forward_ok(w, types[0], 1.0, 0.0)
    backward_ok(w, window(r_out), 1.0, 0.0)


def test_transposed_and_broadcast_rows_are_taken():
    c = make(16, 48, F32, F32, F32)
    c["y"] = c["y"].t().contiguous().t()
    c["dh"] = c["dh"][:1].expand(16, 48)
    c["r"] = c["r"][:1].expand(16, 48)
    r_out, _ = forward_ok(c, F32, 1.0, 0.0)
    backward_ok(c, r_out, 1.0, 0.0)


def test_in_place():
    c = make(50, 512, BF16, F32, F32, gate="token")
    want = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"])
    r = c["r"].clone()
    got = moe.block_norm(r, c["y"], c["w_post"], c["w_pre"], c["gate"], inplace=True)
    assert got[0] is r and torch.equal(r, want[0]) and torch.equal(got[1], want[1])


def test_no_tokens():
    c = make(0, 64, BF16, BF16, BF16, gate="channel")
    r_out, h = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"])
    assert r_out.shape == (0, 64) and h.shape == (0, 64)
    g = moe.block_norm_backward(c["dr_out"], c["dh"], r_out, c["y"], c["w_post"], c["w_pre"], c["gate"])
    for n in ("dw_post", "dw_pre", "dgate"):
        assert g[n].shape == (64,) and not g[n].any()


def test_zero_and_odd_rows():
    """Rows of zeros (only eps under the root), huge and tiny ones, and a row
    of NaN, which stays alone."""
    c = make(6, 128, F32, F32, F32)
    c["r"][0] = c["y"][0] = 0
    c["r"][1] *= 1e12
    c["y"][2] *= 1e-18
    c["y"][3] *= 1e15
    forward_ok(c, F32, 1.0, 0.0)
    c["y"][4, 5] = float("nan")
    c["r"][5, 7] = float("inf")
    r_out, h = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"])
    assert torch.isnan(h[4]).all() and torch.isfinite(h[:4]).all() and torch.isnan(h[5, 7])


@pytest.mark.parametrize("T,H", [(1, 64), (3, 64), (33, 40), (5, 7), (10001, 256), (10001, 77), (4865, 2048)])
@pytest.mark.parametrize("gate", ["none", "channel"])
def test_infinite_gradients_are_not_lost(T, H, gate):
    """An infinite gradient of one channel makes that channel's weight gradient
    infinite, whatever the number of rows (blocks that rows do not fill have
    others in their places, which add nothing)."""
    c = make(T, H, F32, F32, F32, gate=gate, seed=5)
    r_out, _ = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"])
    for t in {0, T // 2, T - 1}:
        dh, dr = c["dh"].clone(), c["dr_out"].clone()
        dh[t, 5] = INF
        g = moe.block_norm_backward(dr, dh, r_out, c["y"], c["w_post"], c["w_pre"], c["gate"])
        want = INF if r_out[t, 5] > 0 else -INF
        assert g["dw_pre"][5] == want and torch.isfinite(torch.cat([g["dw_pre"][:5], g["dw_pre"][6:]])).all()
        dr[t, 3] = INF
        g = moe.block_norm_backward(dr, c["dh"], r_out, c["y"], c["w_post"], c["w_pre"], c["gate"])
        assert torch.isinf(g["dw_post"][3]) and torch.isfinite(g["dw_post"][4:]).all()
        assert gate == "none" or (torch.isinf(g["dgate"][3]) and torch.isfinite(g["dgate"][4:]).all())


@pytest.mark.parametrize("types,H", [(TYPES[0], 1001), (TYPES[1], 2048), (TYPES[2], 64), (TYPES[1], 77)])
def test_rows_do_not_depend_on_the_batch(types, H):
    c = make(777, H, *types, gate="token")
    full = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"])
    g = moe.block_norm_backward(c["dr_out"], c["dh"], full[0], c["y"], c["w_post"], c["w_pre"], c["gate"])
    for rows in (slice(0, 1), slice(5, 6), slice(100, 333), slice(776, 777)):
        part = moe.block_norm(c["r"][rows], c["y"][rows], c["w_post"], c["w_pre"], c["gate"][rows])
        assert torch.equal(part[0], full[0][rows]) and torch.equal(part[1], full[1][rows])
        p = moe.block_norm_backward(c["dr_out"][rows], c["dh"][rows], full[0][rows], c["y"][rows], c["w_post"],
                                    c["w_pre"], c["gate"][rows])
        for n in ("dr", "dy", "dgate"):
            assert torch.equal(p[n], g[n][rows]), n
    again = moe.block_norm_backward(c["dr_out"], c["dh"], full[0], c["y"], c["w_post"], c["w_pre"], c["gate"])
    assert all(torch.equal(again[n], g[n]) for n in g)


@pytest.mark.parametrize("types,H,ld", [(TYPES[0], 77, 80), (TYPES[1], 77, 78), (TYPES[2], 100, 101), (TYPES[1], 264, 267),
                                        (TYPES[1], 2048, 2051), (TYPES[0], 2048, 2056)])
def test_strided_rows_do_not_depend_on_the_batch(types, H, ld):
    """One row of a strided batch, too, which torch takes for a contiguous one."""
    w, window = windows(make(300, H, *types, gate="element"), ld, 0)
    full = moe.block_norm(w["r"], w["y"], w["w_post"], w["w_pre"], w["gate"])
    r_out = window(full[0])
    g = moe.block_norm_backward(w["dr_out"], w["dh"], r_out, w["y"], w["w_post"], w["w_pre"], w["gate"])
    for rows in (slice(0, 1), slice(5, 6), slice(8, 9), slice(100, 133), slice(299, 300)):
        part = moe.block_norm(w["r"][rows], w["y"][rows], w["w_post"], w["w_pre"], w["gate"][rows])
        assert torch.equal(part[0], full[0][rows]) and torch.equal(part[1], full[1][rows])
        p = moe.block_norm_backward(w["dr_out"][rows], w["dh"][rows], r_out[rows], w["y"][rows], w["w_post"], w["w_pre"],
                                    w["gate"][rows])
        assert all(torch.equal(p[n], g[n][rows]) for n in ("dr", "dy", "dgate"))
    d = dict(w, y=w["y"].contiguous(), gate=w["gate"].contiguous())  # strided residual rows alone: what comes out is dense
    full = moe.block_norm(d["r"], d["y"], d["w_post"], d["w_pre"], d["gate"])
    args = (d["w_post"], d["w_pre"])
    g = moe.block_norm_backward(full[0], full[1], full[0], d["y"], *args, d["gate"])
    for rows in (slice(5, 6), slice(8, 10)):
        part = moe.block_norm(d["r"][rows], d["y"][rows], *args, d["gate"][rows])
        assert all(torch.equal(a, b[rows]) and a.stride() == (H, 1) for a, b in zip(part, full))
        p = moe.block_norm_backward(part[0], part[1], part[0], d["y"][rows], *args, d["gate"][rows])
        assert all(torch.equal(p[n], g[n][rows]) and p[n].stride() == (H, 1) for n in ("dr", "dy", "dgate"))


@pytest.mark.parametrize("types,H", [(TYPES[1], 2048), (TYPES[2], 256), (TYPES[0], 333)])
def test_rows_of_a_large_batch_are_those_of_a_small_one(types, H):
    """Large batches take several rows at a time: the same bits all the same."""
    c = make(20001, H, *types, gate="element")
    full = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"])
    g = moe.block_norm_backward(c["dr_out"], c["dh"], full[0], c["y"], c["w_post"], c["w_pre"], c["gate"])
    for rows in (slice(0, 3), slice(7777, 7790), slice(20000, 20001)):
        part = moe.block_norm(c["r"][rows], c["y"][rows], c["w_post"], c["w_pre"], c["gate"][rows])
        assert torch.equal(part[0], full[0][rows]) and torch.equal(part[1], full[1][rows])
        p = moe.block_norm_backward(c["dr_out"][rows], c["dh"][rows], full[0][rows], c["y"][rows], c["w_post"],
                                    c["w_pre"], c["gate"][rows])
        assert all(torch.equal(p[n], g[n][rows]) for n in ("dr", "dy", "dgate"))


def test_gradients_against_differences():
    """Central differences of sum(a r_out + b h) along random directions.  The
    loss is summed in 64 bits; with step 1e-2 the cut-off error is of order
    1e-4 of the derivative's terms and the outputs' roundings, 2^-24 of each
    over the step, are below that."""
    T, H = 11, 200
    c = make(T, H, F32, F32, F32, gate="element")
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b = torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda")

    def loss(d):
        r_out, h = moe.block_norm(d["r"], d["y"], d["w_post"], d["w_pre"], d["gate"], scale=0.7)
        return float((a.double() * r_out.double()).sum() + (b.double() * h.double()).sum())

    r_out, _ = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], c["gate"], scale=0.7)
    grad = moe.block_norm_backward(a, b, r_out, c["y"], c["w_post"], c["w_pre"], c["gate"], scale=0.7)
    for name, key in (("r", "dr"), ("y", "dy"), ("w_post", "dw_post"), ("w_pre", "dw_pre"), ("gate", "dgate")):
        v = torch.randn(c[name].shape, generator=g, device="cuda")
        step = 1e-2
        num = (loss(dict(c, **{name: c[name] + step * v})) - loss(dict(c, **{name: c[name] - step * v}))) / (2 * step)
        terms = (grad[key].double() * v.double())
        assert abs(num - float(terms.sum())) <= 2e-3 * float(terms.abs().sum()), name


def test_side_stream():
    c = make(64, 1024, BF16, BF16, BF16)
    want = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], stream=s)
    g = moe.block_norm_backward(c["dr_out"], c["dh"], got[0], c["y"], c["w_post"], c["w_pre"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    w = moe.block_norm_backward(c["dr_out"], c["dh"], want[0], c["y"], c["w_post"], c["w_pre"])
    assert all(g[n] is None or torch.equal(g[n], w[n]) for n in g)


@pytest.mark.parametrize("T,H,ld", [(4, 64, 64), (3000, 77, 77), (3000, 77, 80), (20000, 3, 4), (20, 4104, 4104), (700, 2048, 2056)])
def test_a_workspace_asked_for_without_buffers(T, H, ld):
    """Its size is that of the call, and the call takes it."""
    from top_routed_grouped_gb300 import step
    size = step.moe_block_norm_workspace_size(step._NORM.pack(T, H, 1, 1, 1, 3, 1.0, EPS, 0.0, 0, *[ld] * 10, *[0] * 14))
    assert size >= 3 * H * 4 and size % 256 == 0
    c = make(T, H, BF16, BF16, BF16, gate="element")
    w, window = windows(c, ld, 0)
    r_out = window(forward_ok(w, BF16, 1.0, 0.0)[0])
    args = (w["dr_out"], w["dh"], r_out, w["y"], w["w_post"], w["w_pre"], w["gate"])
    want = moe.block_norm_backward(*args)
    got = moe.block_norm_backward(*args, ws=torch.empty(size, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_refusals():
    c = make(4, 64, BF16, F32, F32)
    ok = lambda **k: moe.block_norm(**dict(dict(r=c["r"], y=c["y"], w_post=c["w_post"], w_pre=c["w_pre"]), **k))  # noqa: E731
    ok()
    for bad in (dict(y=c["y"][:3]), dict(y=c["y"].half()), dict(r=c["r"].to(BF16).half()), dict(w_post=c["w_post"][:5]),
                dict(w_post=c["w_post"].to(BF16)), dict(gate=torch.ones(4, 2, device="cuda")),
                dict(gate=torch.ones(4, 1, device="cuda", dtype=BF16)), dict(y=None), dict(r=c["r"].cpu()),
                dict(y=None, w_post=None, w_pre=None)):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(moe.MoEError):
        ok(eps=-1.0)
    with pytest.raises(moe.MoEError):
        ok(scale=float("nan"))
    wide = torch.ones(2, 16392, device="cuda")
    with pytest.raises(moe.MoEError) as e:
        moe.block_norm(wide, None, None, wide[0])
    assert e.value.status == -2
    with pytest.raises(moe.MoEError) as e:
        moe.block_norm_backward(c["dr_out"], c["dh"], c["r"], c["y"], c["w_post"], c["w_pre"],
                                ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -3
    with pytest.raises(ValueError):
        moe.block_norm_backward(c["dr_out"], None, c["r"], c["y"], c["w_post"], c["w_pre"])
    with pytest.raises(ValueError):
        moe.block_norm_backward(None, None, None, c["y"], c["w_post"])
