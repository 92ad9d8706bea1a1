"""embed and its gradient by sorted tokens against the plain 64-bit form."""
import pytest
import torch

import _step_ref as ref
import top_routed_grouped_gb300 as moe

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tokens(kind, T, V, seed=0, dtype=torch.int64):
    g = gen(seed)
    if kind == "same":
        ids = torch.full((T,), V // 2, device="cuda")
    elif kind == "ends":
        ids = (V - 1) * torch.randint(2, (T,), generator=g, device="cuda")
    elif kind == "ranks":  # frequencies 1/n
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * torch.log(torch.tensor(float(V), dtype=torch.float64))) - 1).long().clamp(0, V - 1)
    elif kind == "down":
        ids = (V - 1 - torch.arange(T, device="cuda")) % V
    else:
        ids = torch.randint(V, (T,), generator=g, device="cuda")
    return ids.to(dtype)


@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (5, 3, 2), (17, 1000, 7), (64, 50257, 64), (33, 777, 1001),
                                   (300, 4096, 2048), (7, 1048575, 16)])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("itype", [torch.int64, torch.int32])
def test_lookup(T, V, H, dtype, out, itype):
    table = torch.randn(V, H, generator=gen(V), device="cuda").to(dtype)
    ids = tokens("any", T, V, dtype=itype)
    got = moe.embed(table, ids, scale=H ** 0.5, out_dtype=out)
    assert got.dtype == out
    ref.check(got, *ref.embed(table, ids, H ** 0.5), ops=2, what="out")


@pytest.mark.parametrize("kind", ["same", "ends", "ranks", "down", "any"])
@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (2, 5, 3), (31, 1, 64), (1000, 77, 33), (4096, 1025, 128),
                                   (700, 50257, 100), (5000, 3000, 264)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient(kind, T, V, H, dtype):
    ids = tokens(kind, T, V)
    dout = torch.randn(T, H, generator=gen(T), device="cuda").to(dtype)
    got = moe.embed_backward(ids, dout, V, scale=3.0)
    want, mag = ref.embed_backward(ids, dout, V, 3.0)
    ref.check(got, want, mag, ops=T + 8, what="dtable")
    assert torch.equal(got, moe.embed_backward(ids.int(), dout, V, scale=3.0))
    assert not got[want.abs().sum(1) + mag.sum(1) == 0].any()


@pytest.mark.parametrize("T,V,H", [(70000, 131, 40), (65536, 200000, 16), (1 << 20, 5000, 8), ((1 << 20) + 77, 300, 4)])
def test_gradient_of_many_tokens(T, V, H):
    ids = tokens("ranks", T, V)
    dout = torch.randn(T, H, generator=gen(5), device="cuda")
    want, mag = ref.embed_backward(ids, dout, V, 1.0)
    got = moe.embed_backward(ids, dout, V)
    ref.check(got, want, mag, ops=T + 8, what="dtable")
    assert torch.equal(got, moe.embed_backward(ids, dout, V))


@pytest.mark.parametrize("kind", ["same", "ends", "ranks", "any"])
@pytest.mark.parametrize("T,V,H,pad", [(1, 3, 8, 0), (4095, 50, 16, 0), (16385, 1000, 24, 8), (65537, 400, 8, 0), (131072, 900, 8, 0), (131073, 900, 8, 0),
                                       (131073, 70000, 12, 5), (200000, 33, 16, 16), (262145, 1025, 9, 0), (300000, 1 << 19, 8, 3),
                                       ((1 << 20) - 1, 5000, 8, 0), ((1 << 20) + 77, 2100, 7, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_whole_numbers_are_summed_exactly(kind, T, V, H, pad, dtype):
    """Gradients of small whole numbers: every sum in FP32 is exact (below 2^24)
    in any order, so a row that is lost, counted twice or given to another
    token shows as a difference.  On both sides of the token counts at which the
    sort and the tiles change; some tokens padding, some outside the table."""
    g = gen(T + V)
    ids = tokens(kind, T, V, seed=V, dtype=torch.int32 if T % 2 else torch.int64)
    ids[::97] = -1
    ids[::89] = V
    dout = torch.randint(-8, 9, (T, H + pad), generator=g, device="cuda").to(dtype)[:, :H]
    first = torch.randint(-8, 9, (V, H), generator=g, device="cuda").float()
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda")
    ok = (ids >= 0) & (ids < V)
    want.index_add_(0, ids[ok].long(), 2.0 * dout[ok].double())
    assert float(want.abs().max()) < 2 ** 24
    moe.moe_device_status(reset=True)
    got = moe.embed_backward(ids, dout, V, scale=2.0)
    assert moe.moe_device_status(reset=True) == 5
    assert torch.equal(got.double(), want)
    token, sums = int(ids[T // 2].clamp(0, V - 1)), first.clone()
    moe.embed_backward(ids, dout, V, scale=2.0, padding_id=token, dtable=sums)
    want[token] = 0
    assert torch.equal(sums.double(), first.double() + want)


@pytest.mark.parametrize("dtype,H", [(F32, 96), (BF16, 72), (BF16, 13)])
def test_padding_bad_ids_and_accumulation(dtype, H):
    T, V = 900, 60
    ids = tokens("any", T, V + 20) - 10  # some below 0, some past the table
    dout = torch.randn(T, H, generator=gen(9), device="cuda").to(dtype)
    dout[ids == 7] = float("nan")  # the padding token's rows are not read
    moe.moe_device_status(reset=True)
    got = moe.embed_backward(ids, dout, V, scale=0.5, padding_id=7)
    assert moe.moe_device_status(reset=True) == 5
    want, mag = ref.embed_backward(ids, dout, V, 0.5, padding_id=7)
    ref.check(got, want, mag, ops=T + 8, what="dtable")
    assert not got[7].any()
    first = torch.randn(V, H, generator=gen(10), device="cuda")
    hit = mag.sum(1) > 0
    acc = first.clone()
    assert moe.embed_backward(ids, dout, V, scale=0.5, padding_id=7, dtable=acc) is acc
    ref.check(acc, first.double() + want, first.abs().double() + mag, ops=T + 9, what="accumulated")
    assert torch.equal(acc[~hit], first[~hit])
    moe.moe_device_status(reset=True)
    table = torch.randn(V, H, generator=gen(11), device="cuda").to(dtype)
    out = moe.embed(table, ids)
    assert moe.moe_device_status(reset=True) == 5
    bad = (ids < 0) | (ids >= V)
    assert not out[bad].any()
    ref.check(out, *ref.embed(table, ids, 1.0), ops=2, what="out")


def test_all_left_out():
    ids = torch.full((40,), 3, device="cuda")
    got = moe.embed_backward(ids, torch.full((40, 24), float("nan"), device="cuda"), 9, padding_id=3)
    assert got.shape == (9, 24) and not got.any()


def test_no_tokens():
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    dout = torch.empty(0, 16, device="cuda")
    assert not moe.embed_backward(ids, dout, 50).any()
    keep = torch.ones(50, 16, device="cuda")
    assert torch.equal(moe.embed_backward(ids, dout, 50, dtable=keep), torch.ones(50, 16, device="cuda"))
    assert moe.embed(torch.ones(5, 16, device="cuda"), ids).shape == (0, 16)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 2), (4, 4)])
def test_strided_rows(dtype, shift, pad):
    V, H, T = 300, 120, 257
    ids = tokens("ranks", T, V)
    wide = torch.randn(V, H + shift + pad, generator=gen(1), device="cuda").to(dtype)
    table = wide[:, shift:shift + H]
    ref.check(moe.embed(table, ids, 2.0), *ref.embed(table, ids, 2.0), ops=2, what="out")
    d = torch.randn(T, H + shift + pad, generator=gen(2), device="cuda").to(dtype)[:, shift:shift + H]
    ref.check(moe.embed_backward(ids, d, V), *ref.embed_backward(ids, d, V, 1.0), ops=T + 8, what="dtable")
    every = d[:1].expand(T, H)
    ref.check(moe.embed_backward(ids, every, V), *ref.embed_backward(ids, every, V, 1.0), ops=T + 8, what="broadcast")


def test_gradient_against_differences():
    """The lookup is linear in the table: a difference quotient of any step is
    the directional derivative, up to the roundings (2^-24 of each term)."""
    V, H, T = 40, 24, 200
    ids = tokens("ranks", T, V)
    table, a = torch.randn(V, H, generator=gen(1), device="cuda"), torch.randn(T, H, generator=gen(2), device="cuda")
    v = torch.randn(V, H, generator=gen(3), device="cuda")
    f = lambda w: float((moe.embed(w, ids, 1.5).double() * a.double()).sum())  # noqa: E731
    num = (f(table + v) - f(table - v)) / 2
    terms = moe.embed_backward(ids, a, V, 1.5).double() * v.double()
    assert abs(num - float(terms.sum())) <= 1e-5 * float(terms.abs().sum())


def test_table_past_32_bit_offsets():
    """Rows whose element offsets pass 2^31."""
    V, H = 300000, 8192
    table = torch.zeros(V, H, dtype=BF16, device="cuda")
    table[V - 1] = 2.0
    table[270000] = 3.0
    ids = torch.tensor([V - 1, 0, 270000], device="cuda")
    out = moe.embed(table, ids)
    assert (out[0] == 2).all() and not out[1].any() and (out[2] == 3).all()
    del table
    d = moe.embed_backward(ids, out, V)
    assert (d[V - 1] == 2).all() and (d[270000] == 3).all() and int((d != 0).sum()) == 2 * H


def test_side_stream():
    ids = tokens("ranks", 3000, 500)
    dout = torch.randn(3000, 256, generator=gen(1), device="cuda")
    want = moe.embed_backward(ids, dout, 500)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.embed_backward(ids, dout, 500, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


def test_refusals():
    table, ids = torch.ones(10, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    dout = torch.ones(4, 8, device="cuda")
    for f in (lambda: moe.embed(table.half(), ids), lambda: moe.embed(table, ids.float()),
              lambda: moe.embed(table, ids[None]), lambda: moe.embed(table, ids.cpu()),
              lambda: moe.embed(table, ids, out_dtype=BF16), lambda: moe.embed(table.cpu(), ids),
              lambda: moe.embed_backward(ids[:3], dout, 10),
              lambda: moe.embed_backward(ids, dout, 10, dtable=torch.ones(10, 8, device="cuda", dtype=BF16)),
              lambda: moe.embed_backward(ids, dout, 10, dtable=torch.ones(9, 8, device="cuda"))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(moe.MoEError) as e:
        moe.embed_backward(ids, dout, 1 << 20)
    assert e.value.status == -2
    with pytest.raises(moe.MoEError) as e:
        moe.embed_backward(ids, dout, 10, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -3
    with pytest.raises(moe.MoEError):
        moe.embed(table, ids, scale=float("inf"))
