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
