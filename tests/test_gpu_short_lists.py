"""Norms of lists so short that most CTAs of a cluster have nothing to read: they
meet the one that adds up before they write to it."""
import pytest
import torch

import top_routed_grouped_gb300 as moe
from test_gpu_grads import NORM_TOL, make, near, norm64

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("sizes", [[1], [3], [8192], [8193], [1, 1], [5000, 1, 7], [8192] * 9], ids=str)
@pytest.mark.parametrize("dtype", [F, B])
def test_many_short_lists_one_after_another(sizes, dtype):
    ts = make(sizes, (dtype,))
    want = norm64(ts)
    norms = [moe.grad_norm(ts) for _ in range(300)]
    clips = [moe.clip_grads(ts, 2 * want + 1) for _ in range(100)]
    near(norms[0], want, NORM_TOL)
    assert all(torch.equal(n, norms[0]) for n in norms + clips)


@pytest.mark.parametrize("dtype", [F, B])
def test_bits_go_by_the_addresses_modulo_16(dtype):
    """Moved by whole 16 bytes the same gradients have the same norm; by less they have it to its bound."""
    sizes = [40003, 7, 8192, 100001]
    at = make(sizes, (dtype,))
    unit = 16 // at[0].element_size()

    def moved(by):
        out = []
        for t in at:
            flat = torch.empty(t.numel() + by, device="cuda", dtype=dtype)
            flat[by:] = t
            out.append(flat[by:])
        return out

    for by in (1, 2, 3):
        first = moved(by)
        assert torch.equal(moe.grad_norm(moved(by + unit)), moe.grad_norm(first))
        assert torch.equal(moe.grad_norm(moved(by + 5 * unit)), moe.grad_norm(first))
        near(moe.grad_norm(first), norm64(at), NORM_TOL)


def test_an_infinite_max_norm_reads_the_norm():
    """As with the function of torch whose name it bears."""
    ps = [torch.nn.Parameter(torch.zeros(n, device="cuda", dtype=t)) for n, t in ((300, F), (70, B), (5, F))]
    ps[0].grad, ps[1].grad = make([300, 70], (F, B))
    before = [p.grad.clone() for p in ps[:2]]
    versions = [p.grad._version for p in ps[:2]]
    assert torch.equal(moe.clip_grad_norm_(ps, float("inf")), moe.grad_norm(before))
    assert all(torch.equal(p.grad, b) for p, b in zip(ps, before)) and versions == [p.grad._version for p in ps[:2]]
    ps[0].grad[7] = float("nan")
    assert torch.isnan(moe.clip_grad_norm_(iter(ps), float("inf"))) and torch.equal(ps[1].grad, before[1])
    for bad in (float("-inf"), float("nan"), -1.0):
        with pytest.raises(moe.MoEError):
            moe.clip_grad_norm_(ps, bad)
