"""Host-side checks of the end of a training step (no GPU work): packed structs
match the header, bad arguments return an error and launch nothing."""
import ctypes
import re
from array import array

import pytest
import torch

import top_routed_grouped_gb300 as moe
from test_step_host import PTR, L, fields, packed  # noqa: F401
from top_routed_grouped_gb300 import train


@pytest.mark.parametrize("name,spec", [("moe_linear_ce_args", train._CE), ("moe_grads_args", train._GRADS)])
def test_structs_match_the_header(name, spec):
    f = fields(name)
    assert "".join(k for _, k in f) == re.sub(r"(\d+)(\w)", lambda m: int(m.group(1)) * m.group(2), spec.format)
    cls = type("S", (ctypes.Structure,), {"_fields_": [
        (n, {"i": ctypes.c_int32, "f": ctypes.c_float, "q": ctypes.c_int64, "Q": ctypes.c_void_p}[k]) for n, k in f]})
    assert ctypes.sizeof(cls) == spec.size


def ce(**kw):
    return packed("moe_linear_ce_args", train._CE,
                  **dict(dict(T=4, D=64, V=100, dtype=1, dweight_dtype=1, scale=1.0, ignore_index=-100), **kw))


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), -1), (dict(D=0), -1), (dict(V=0), -1), (dict(D=16385), -2), (dict(V=(1 << 20) + 1), -2),
    (dict(T=(1 << 24) + 1), -2), (dict(dtype=2), -1), (dict(dweight_dtype=7), -1), (dict(dtype=0, dweight_dtype=1), -1),
    (dict(accumulate=1), -1), (dict(accumulate=2, dweight_dtype=0), -1), (dict(targets64=2), -1), (dict(reserved=1), -1),
    (dict(scale=float("inf")), -1), (dict(scale=float("nan")), -1), (dict(z_loss=-0.1), -1), (dict(z_loss=float("nan")), -1),
    (dict(ld_hidden=63), -1), (dict(ld_weight=-64), -1), (dict(ld_dhidden=1), -1), (dict(hidden=0), -1),
    (dict(hidden=PTR + 1), -1), (dict(weight=0), -1), (dict(weight=PTR + 1), -1), (dict(targets=0), -1),
    (dict(targets=PTR + 2), -1), (dict(targets64=1, targets=PTR + 4), -1), (dict(loss=0), -1), (dict(loss=PTR + 2), -1),
    (dict(lse=0), -1),
])
def test_loss_refusals(L, kw, want):  # noqa: F811
    assert L.moe_linear_ce(ce(**kw), PTR, 1 << 40, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dhidden=0), -1), (dict(dhidden=PTR + 1), -1), (dict(dweight=0), -1), (dict(dweight=PTR + 1), -1),
    (dict(dweight_dtype=0, dweight=PTR + 2), -1), (dict(dloss=0), -1), (dict(dloss=PTR + 1), -1), (dict(lse=PTR + 2), -1),
    (dict(T=0, dweight=0), -1),
])
def test_gradient_refusals(L, kw, want):  # noqa: F811
    assert L.moe_linear_ce_backward(ce(**kw), PTR, 1 << 40, None) == want
    assert L.moe_linear_ce_step(ce(**kw), PTR, 1 << 40, None) == want


def test_lse_of_the_gradient_and_of_the_step(L):  # noqa: F811
    assert L.moe_linear_ce_backward(ce(lse=0), PTR, 1 << 40, None) == -1
    assert L.moe_linear_ce_step(ce(lse=0), PTR, 0, None) == -3  # (the step may leave it out: the workspace is next)


def test_missing_arguments(L):  # noqa: F811
    assert L.moe_linear_ce(None, None, 0, None) == -1 and L.moe_linear_ce_workspace_size(None, 1) == 0
    assert L.moe_grad_norm(None, None, 0, None) == -1 and L.moe_grad_scale(None, None) == -1
    assert L.moe_grad_workspace_size(None) == 0


@pytest.mark.parametrize("T,D,V", [(1, 1, 1), (4, 64, 100), (5000, 77, 50257), (8192, 2048, 131072), (100000, 64, 1000)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_workspace_goes_by_sizes(L, T, D, V, dtype):  # noqa: F811
    """One size whether the buffers are there or not; a short one and a misaligned one are refused."""
    kw = dict(T=T, D=D, V=V, dtype=dtype, dweight_dtype=dtype)
    none = {n: 0 for n, k in fields("moe_linear_ce_args") if k == "Q"}
    for call, f in ((1, L.moe_linear_ce), (2, L.moe_linear_ce_backward), (3, L.moe_linear_ce_step)):
        n = L.moe_linear_ce_workspace_size(ce(**kw), call)
        assert n > 0 and n % 256 == 0 and n == L.moe_linear_ce_workspace_size(ce(**dict(kw, **none)), call)
        assert f(ce(**kw), PTR, n - 1, None) == -3
        assert f(ce(**kw), 0, n, None) == -1 and f(ce(**kw), PTR + 16, n, None) == -1
        assert L.moe_linear_ce_workspace_size(ce(**dict(kw, ld_weight=D + 1)), call) >= n
    assert L.moe_linear_ce_workspace_size(ce(T=0), 3) == 0
    assert L.moe_linear_ce_workspace_size(ce(**kw), 0) == 0 and L.moe_linear_ce_workspace_size(ce(**kw), 4) == 0
    assert n < 6 << 30  # g of a piece, not of the vocabulary


def grads(ranges, outs=None, **kw):
    """(address, elements, type) of each tensor -> the packed struct and what keeps its arrays alive."""
    a = [array("Q", [r[0] for r in ranges]), array("Q", [r[0] for r in (outs or ranges)]),
         array("q", [r[1] for r in ranges]), array("i", [r[2] for r in ranges]),
         array("i", [r[2] for r in (outs or ranges)])]
    base = dict(n=len(ranges), reserved=0, max_norm=1.0, eps=0.0, norm=PTR,
                **dict(zip(("in", "out", "numel", "dtype", "odtype"), (x.buffer_info()[0] for x in a))))
    base.update(kw)
    return train._GRADS.pack(*[base[n] for n in ("n", "reserved", "in", "out", "numel", "dtype", "odtype", "max_norm",
                                                 "eps", "norm")]), a


M = 1 << 20


@pytest.mark.parametrize("ranges,kw,want", [
    ([(M, 4, 0)], dict(n=-1), -1), ([(M, 4, 0)], dict(n=(1 << 20) + 1), -2), ([(M, 4, 0)], dict(reserved=3), -1),
    ([(M, -1, 0)], {}, -1), ([(M, 4, 2)], {}, -1), ([(0, 4, 0)], {}, -1), ([(M + 2, 4, 0)], {}, -1),
    ([(M + 1, 4, 1)], {}, -1), ([(M, (1 << 42) + 1, 1)], {}, -2), ([(M, 1 << 41, 1)] * 3, {}, -2),
    ([(M, 4, 0)], dict(norm=0), -1), ([(M, 4, 0)], dict(norm=PTR + 2), -1), ([(M, 4, 0)], {"in": 0}, -1),
    ([(M, 4, 0)], dict(numel=0), -1), ([(M, 4, 0)], dict(dtype=0), -1),
])
def test_norm_refusals(L, ranges, kw, want):  # noqa: F811
    args, keep = grads(ranges, **kw)
    assert L.moe_grad_norm(args, PTR, 1 << 30, None) == want
    assert L.moe_grad_clip(args, PTR, 1 << 30, None) == want


@pytest.mark.parametrize("ranges,out,kw", [
    ([(M, 4, 0)], None, dict(max_norm=-1.0)), ([(M, 4, 0)], None, dict(max_norm=float("inf"))),
    ([(M, 4, 0)], None, dict(max_norm=float("nan"))), ([(M, 4, 0)], None, dict(eps=-1.0)), ([(M, 4, 0)], None, dict(out=0)),
    ([(M, 4, 0)], None, dict(odtype=0)), ([(M, 4, 0)], [(M + 64, 4, 3)], {}), ([(M, 4, 0)], [(0, 4, 0)], {}),
    ([(M, 4, 0)], [(M + 65, 4, 1)], {}),
    ([(M, 8, 0), (M + 16, 8, 0)], None, {}),                               # tensors over one another
    ([(M, 8, 0), (M, 8, 0)], None, {}),                                    # one of them twice
    ([(M, 8, 0)], [(M + 4, 8, 0)], {}),                                    # an output over its own input, shifted
    ([(M, 8, 0)], [(M, 8, 1)], {}),                                        # ... in another type
    ([(M, 8, 0), (M + 32, 8, 0)], [(M + 64, 8, 0), (M, 8, 0)], {}),        # over another's input
    ([(M, 8, 0), (M + 32, 8, 0)], [(M + 64, 8, 0), (M + 80, 8, 0)], {}),   # outputs over one another
    ([(M + 64, 64, 0), (M, 8, 0)], [(2 * M, 64, 0), (M + 128, 8, 0)], {}),  # inside a longer input
])
def test_clip_refusals(L, ranges, out, kw):  # noqa: F811
    args, keep = grads(ranges, out, **kw)
    assert L.moe_grad_clip(args, PTR, 1 << 30, None) == -1
    assert L.moe_grad_scale(args, None) == -1


def test_tensors_on_the_host_are_refused():
    t = torch.zeros(3, 4)
    for f in (lambda: moe.linear_cross_entropy(t, t, torch.zeros(3, dtype=torch.int64)), lambda: moe.grad_norm([t]),
              lambda: moe.clip_grads([t], 1.0), lambda: moe.scale_grads([t], torch.ones(()), 1.0),
              lambda: moe.grad_norm([None]), lambda: moe.clip_grads([1.0], 1.0)):
        with pytest.raises(ValueError):
            f()
