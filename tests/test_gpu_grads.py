"""grad_norm, clip_grads and scale_grads against 64 bits.

The norm: squares in FP32 (2^-24 each), at most 34 of them a thread in sums of
FP32 (4 chains and their joining: 12 roundings, then 5 of a warp's tree), the
rest in FP64, the root halves it, one rounding to float: below 16 * 2^-24 relative.  A scaled element: the factor's own
few roundings (the norm's, the sum with eps, the quotient: 20 * 2^-24), the
product, and half an ulp of the output's type (2^-8, 2^-24)."""
import pytest
import torch

import top_routed_grouped_gb300 as moe

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16
U = {F: 2.0 ** -24, B: 2.0 ** -8}
NORM_TOL, SCALE_TOL = 16 * 2.0 ** -24, 24 * 2.0 ** -24


def make(sizes, dtypes, seed=0, size=1.0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        x = (torch.randn(n + shift, generator=g, device="cuda") * size).to(dtypes[i % len(dtypes)])
        out.append(x[shift:])
    return out


def norm64(ts):
    return float(torch.stack([t.double().square().sum() for t in ts]).sum().sqrt())


def near(got, want, tol):
    assert abs(float(got) - want) <= tol * abs(want) + 1e-45, (float(got), want)


def clipped_ok(outs, before, norm, max_norm, eps=1e-6):
    c = min(1.0, max_norm / (norm + eps))
    for o, b in zip(outs, before):
        want = b.double() * c
        assert bool(((o.double() - want).abs() <= (SCALE_TOL + U[o.dtype]) * want.abs() + 1e-40).all())


SIZES = [[1], [7], [8], [9], [31, 1, 8192], [8191], [8193, 5], [16384, 8192, 3], [0, 5, 0], [1] * 70, [3, 0, 100003, 17],
         [1000] * 1100, [257] * 2100 + [100000], [3_000_001]]


@pytest.mark.parametrize("dtypes", [(F,), (B,), (F, B)])
@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}of{sum(s)}")
def test_norm_and_clip(sizes, shift, dtypes):
    ts = make(sizes, dtypes, shift=shift)
    want = norm64(ts)
    near(moe.grad_norm(ts), want, NORM_TOL)
    before = [t.clone() for t in ts]
    for max_norm in (want * 0.3, want * 3):
        outs = [torch.full_like(t, 7) for t in ts]
        near(moe.clip_grads(ts, max_norm, out=outs), want, NORM_TOL)
        clipped_ok(outs, before, want, max_norm)
    assert all(torch.equal(t, b) for t, b in zip(ts, before))
    near(moe.clip_grads(ts, want * 3), want, NORM_TOL)  # nothing to do
    assert all(torch.equal(t, b) for t, b in zip(ts, before))
    near(moe.clip_grads(ts, want * 0.3), want, NORM_TOL)
    clipped_ok(ts, before, want, want * 0.3)


@pytest.mark.parametrize("src,dst", [(F, B), (B, F), (F, F), (B, B)])
@pytest.mark.parametrize("a,b", [(0, 0), (1, 0), (0, 1), (3, 2)])
def test_into_tensors_of_another_type_and_alignment(src, dst, a, b):
    n = 40_003
    base = torch.randn(n + a, device="cuda").to(src)
    out = torch.empty(n + b + 8, device="cuda", dtype=dst).fill_(5)
    ts, outs = [base[a:]], [out[b:b + n]]
    want = norm64(ts)
    moe.clip_grads(ts, 1.0, out=outs)
    clipped_ok(outs, ts, want, 1.0)
    assert bool((out[:b] == 5).all()) and bool((out[b + n:] == 5).all())


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e-18, 1e-12, 1e12, 1e18, 1e25, 1e30])
@pytest.mark.parametrize("dtype", [F, B])
def test_squares_that_float_cannot_hold(size, dtype):
    ts = make([5000, 20000, 3], (dtype,), size=size)
    ts.append(torch.zeros(30000, device="cuda", dtype=dtype))
    near(moe.grad_norm(ts), norm64(ts), NORM_TOL)
    mixed = ts + make([10000], (dtype,), size=min(size * 1e6, 1e31))
    near(moe.grad_norm(mixed), norm64(mixed), NORM_TOL)
    assert float(moe.grad_norm([torch.zeros(9999, device="cuda", dtype=dtype)])) == 0.0


@pytest.mark.parametrize("dtype", [F, B])
def test_norms_that_are_not_finite(dtype):
    for bad in (float("inf"), float("-inf"), float("nan")):
        ts = make([100, 9000], (dtype,))
        ts[1][8500] = bad
        norm = moe.grad_norm(ts)
        assert torch.isnan(norm) if bad != bad else norm == float("inf")
        outs = [torch.empty_like(t) for t in ts]
        moe.clip_grads(ts, 1.0, out=outs)
        if bad != bad:
            assert all(bool(torch.isnan(o).all()) for o in outs)
        else:
            assert not outs[0].any() and torch.isnan(outs[1][8500]) and int((outs[1] != 0).sum()) == 1
    huge = torch.full((100000,), 3e38, device="cuda", dtype=dtype)  # above what a float holds
    assert float(moe.grad_norm([huge])) == float("inf")


def test_orders_in_memory_and_gaps():
    a = torch.randn(40, 30, 20, device="cuda").permute(2, 0, 1)
    b = torch.randn(64, 64, device="cuda").t()
    want = norm64([a, b])
    near(moe.grad_norm([a, b]), want, NORM_TOL)
    before = [a.clone(), b.clone()]
    outs = [torch.empty_like(a), torch.empty_like(b)]
    assert outs[0].stride() == a.stride()
    moe.clip_grads([a, b], 1.0, out=outs)
    clipped_ok(outs, before, want, 1.0)
    moe.clip_grads([a, b], 1.0)
    clipped_ok([a, b], before, want, 1.0)
    for bad in (torch.randn(8, 16, device="cuda")[:, :4], torch.randn(4, 1, device="cuda").expand(4, 4)):
        with pytest.raises(ValueError):
            moe.grad_norm([bad])
    with pytest.raises(ValueError):  # another order of the elements
        moe.clip_grads([b], 1.0, out=[torch.empty(64, 64, device="cuda")])


def test_parts_of_a_norm():
    """What ranks do: the norms of two parts, put together, then each scales its own."""
    ts = make([1000, 77, 30001], (F, B))
    want = norm64(ts)
    parts = torch.stack([moe.grad_norm(ts[:1]), moe.grad_norm(ts[1:])])
    norm = parts.square().sum().sqrt()
    before = [t.clone() for t in ts]
    version = ts[0]._version
    moe.scale_grads(ts[:1], norm, 2.0)
    moe.scale_grads(ts[1:], norm.reshape(1), 2.0)
    assert ts[0]._version > version
    clipped_ok(ts, before, want, 2.0)
    outs = [torch.empty_like(t) for t in before]
    moe.scale_grads(before, norm, 2.0, out=outs)
    clipped_ok(outs, before, want, 2.0)
    moe.scale_grads([], norm, 2.0)


@pytest.mark.parametrize("eps,max_norm", [(0.0, 0.5), (1.0, 0.5), (1e-6, 0.0)])
def test_eps_and_max_norm(eps, max_norm):
    ts = make([100, 20], (F,))
    want, before = norm64(ts), [t.clone() for t in ts]
    moe.clip_grads(ts, max_norm, eps=eps)
    clipped_ok(ts, before, want, max_norm, eps)


def test_the_same_bits_every_time_and_in_place_as_outside():
    ts = make([100001, 33, 7000], (F, B), shift=1)
    outs = [torch.empty_like(t) for t in ts]
    norms = [moe.clip_grads(ts, 1.0, out=outs) for _ in range(3)]
    assert all(torch.equal(n, norms[0]) for n in norms)
    moe.clip_grads(ts, 1.0)
    assert all(torch.equal(a, b) for a, b in zip(ts, outs))


def test_past_32_bits():
    n = (1 << 31) + 12345
    t = torch.zeros(n, device="cuda", dtype=B)
    t[-1], t[0], t[1 << 31] = 3.0, 4.0, 12.0
    near(moe.grad_norm([t]), 13.0, NORM_TOL)
    moe.clip_grads([t], 6.5, eps=0.0)
    assert [float(t[i]) for i in (-1, 0, 1 << 31)] == [1.5, 2.0, 6.0] and int((t != 0).sum()) == 3


def test_empty_lists_streams_and_workspaces():
    assert float(moe.grad_norm([])) == 0.0 and float(moe.clip_grads([], 1.0)) == 0.0
    nothing = [torch.empty(0, device="cuda"), torch.empty(0, 5, device="cuda", dtype=B)]
    assert float(moe.grad_norm(nothing)) == 0.0 and float(moe.clip_grads(nothing, 1.0)) == 0.0
    ts = make([5000, 3], (F,))
    want = moe.grad_norm(ts)
    ws = torch.full((1 << 17,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in (dict(ws=ws), dict(stream=side), dict(stream=side.cuda_stream, ws=ws)):
        got = moe.grad_norm(ts, **kw)
        side.synchronize()
        assert torch.equal(got, want)
    with pytest.raises(moe.MoEError):
        moe.grad_norm(ts, ws=ws[:256])


def test_captured_and_replayed():
    ts = make([70001, 3, 999], (F, B))
    outs = [torch.empty_like(t) for t in ts]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm = moe.clip_grads(ts, 1.0, out=outs)
    for seed in (1, 2):
        for t, n in zip(ts, make([70001, 3, 999], (F, B), seed=seed)):
            t.copy_(n)
        graph.replay()
        want = [torch.empty_like(t) for t in ts]
        assert torch.equal(norm, moe.clip_grads(ts, 1.0, out=want))
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    a = torch.randn(100, device="cuda")
    values = [
        lambda: moe.grad_norm([a.half()]), lambda: moe.grad_norm([a, a.double()]), lambda: moe.grad_norm([a, a.cpu()]),
        lambda: moe.grad_norm([a.cpu()]), lambda: moe.grad_norm([a, None]), lambda: moe.grad_norm([a, a.to_sparse()]),
        lambda: moe.clip_grads([a], 1.0, out=[]), lambda: moe.clip_grads([a], 1.0, out=[a[:50]]),
        lambda: moe.clip_grads([a], 1.0, out=[a.half()]), lambda: moe.scale_grads([a], a.double()[0], 1.0),
        lambda: moe.scale_grads([a], a, 1.0), lambda: moe.scale_grads([a], a[0].cpu(), 1.0),
    ]
    for f in values:
        with pytest.raises(ValueError):
            f()
    before, b = a.clone(), torch.randn(300, device="cuda")
    errors = [  # numbers, and outputs over others
        lambda: moe.clip_grads([a], -1.0), lambda: moe.clip_grads([a], float("nan")), lambda: moe.clip_grads([a], 1.0, eps=-1.0),
        lambda: moe.clip_grads([a], float("inf")), lambda: moe.clip_grads([a, a], 1.0),
        lambda: moe.clip_grads([a[:60], a[40:]], 1.0), lambda: moe.clip_grads([b[:100]], 1.0, out=[b[50:150]]),
        lambda: moe.clip_grads([b[:100], b[100:200]], 1.0, out=[b[100:200], b[200:]]),
        lambda: moe.clip_grads([b[:100]], 1.0, out=[b[:50].view(B)]),
    ]
    for f in errors:
        with pytest.raises(moe.MoEError):
            f()
    assert torch.equal(a, before)
    moe.clip_grads([b[:100], b[100:200]], 1e-3, out=[b[:100], b[200:]])  # each beside the others
    near(moe.grad_norm([a, a]), norm64([a, a]), NORM_TOL)                # read twice
    one = torch.empty(100, device="cuda"), torch.empty(100, device="cuda")
    moe.clip_grads([a, a], 1.0, out=one)
    assert torch.equal(*one)
