"""The end of a training step under autograd, with the embedding that it shares
its table with, and the example that runs all of it."""
import importlib.util
import os

import pytest
import torch

import top_routed_grouped_gb300 as moe
from _train_ref import IGNORE, check, cross_entropy

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F, B])
def test_gradients_under_autograd(dtype):
    T, D, V = 130, 72, 500
    g = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn(T, D, generator=g, device="cuda").to(dtype).requires_grad_()
    w = (torch.randn(V, D, generator=g, device="cuda") * 0.2).to(dtype).requires_grad_()
    t = torch.randint(V, (T,), generator=g, device="cuda")
    t[:17] = IGNORE
    d = torch.rand(T, generator=g, device="cuda")
    loss = moe.cross_entropy_loss(h, w, t, scale=0.5, z_loss=1e-3)
    loss.backward(d)
    ref = cross_entropy(h.detach(), w.detach(), t, d, 0.5, 1e-3)
    check(loss.detach(), ref["loss"], "loss")
    check(h.grad, ref["dhidden"], "dhidden")
    check(w.grad, ref["dweight"], "dweight")
    assert h.grad.dtype is dtype and w.grad.dtype is dtype
    x = torch.randn(4, D, device="cuda").to(dtype).requires_grad_()
    out = moe.cross_entropy_loss(x, w, t[20:24]).sum()
    gx, = torch.autograd.grad(out, x, create_graph=True)
    with pytest.raises(RuntimeError):  # no second derivative
        gx.sum().backward()


def test_dloss_that_is_spread_out():
    """A mean's gradient is one number expanded over the rows."""
    h = torch.randn(64, 64, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(100, 64, device="cuda").bfloat16().requires_grad_()
    t = torch.randint(100, (64,), device="cuda")
    moe.cross_entropy_loss(h, w, t).mean().backward()
    ref = cross_entropy(h.detach(), w.detach(), t, torch.full((64,), 1 / 64, device="cuda"))
    check(h.grad, ref["dhidden"], "dhidden")
    check(w.grad, ref["dweight"], "dweight")


@pytest.mark.parametrize("D", [64, 100])
def test_head_with_the_embeddings_table(D):
    """One table read at both ends: its gradient is the sum of both, clipped with the rest; by the
    modules, and by the calls that add into one float32 tensor."""
    T, V = 90, 300
    g = torch.Generator(device="cuda").manual_seed(4)
    emb = moe.TokenEmbedding(V, D, dtype=F)
    head = moe.LMHead(V, D, weight=emb.weight)
    assert head.weight is emb.weight and len(list(torch.nn.ModuleList([emb, head]).parameters())) == 1
    ids = torch.randint(V, (T,), generator=g, device="cuda")
    targets = torch.randint(V, (T,), generator=g, device="cuda")
    targets[-5:] = IGNORE
    mix = (torch.randn(D, D, generator=g, device="cuda") / D ** 0.5).requires_grad_()
    (head(emb(ids) @ mix, targets).sum() / (T - 5)).backward()
    a = emb.weight.detach().double().requires_grad_()
    b = mix.detach().double().requires_grad_()
    x = torch.nn.functional.cross_entropy(a[ids] @ b @ a.t(), targets, ignore_index=IGNORE)
    x.backward()
    close = lambda p, q: float((p.double() - q).norm()) <= 2e-5 * float(q.norm())  # noqa: E731  (FP32 through a few operators)
    assert close(emb.weight.grad, a.grad) and close(mix.grad, b.grad)
    # The calls themselves: the head's gradient, the embedding's added to it.
    e = moe.embed(emb.weight.detach(), ids)
    total = torch.zeros(V, D, device="cuda")
    d = torch.full((T,), 1 / (T - 5), device="cuda")
    _, dh, _ = moe.linear_cross_entropy_step(e @ mix.detach(), emb.weight.detach(), targets, d, dweight=total)
    moe.embed_backward(ids, dh @ mix.detach().t(), V, dtable=total)
    assert close(total, a.grad)
    want = torch.cat([a.grad.flatten(), b.grad.flatten()]).norm()
    for max_norm in (0.1, 0.01):  # above the norm, and below it
        c = min(1.0, float(max_norm / (want + 1e-6)))
        norm = moe.clip_grad_norm_([emb.weight, mix, torch.nn.Parameter(torch.zeros(3, device="cuda"))], max_norm)
        assert close(norm.reshape(1), want.reshape(1))
        assert close(emb.weight.grad, a.grad * c) and close(mix.grad, b.grad * c)
        assert close(moe.grad_norm([emb.weight.grad, mix.grad]).reshape(1), (want * c).reshape(1))
    assert close(moe.clip_grad_norm_(mix, 1e9).reshape(1), mix.grad.norm().reshape(1))


def test_gradients_of_the_layer_are_handed_on_in_its_type():
    """float32 gradients as the layer's backward leaves them, clipped into bfloat16 ones."""
    grads = [torch.randn(8, 96, 64, device="cuda"), torch.randn(8, 64, 48, device="cuda"), torch.randn(8, 64, device="cuda")]
    outs = [torch.empty_like(x, dtype=B) for x in grads]
    norm = moe.clip_grads(grads, 1.0, out=outs)
    c = min(1.0, 1.0 / (float(norm) + 1e-6))
    for x, o in zip(grads, outs):
        assert bool(((o.double() - x.double() * c).abs() <= (2.0 ** -8 + 2.0 ** -19) * x.double().abs() * c).all())


def test_a_whole_end_of_a_step_captured():
    """Loss, gradients and clipping in one graph, replayed on other rows."""
    T, D, V = 100, 64, 700
    mk = lambda seed: torch.Generator(device="cuda").manual_seed(seed)  # noqa: E731
    data = lambda g: (torch.randn(T, D, generator=g, device="cuda").bfloat16(),  # noqa: E731
                      torch.randint(V, (T,), generator=g, device="cuda"))
    w = (torch.randn(V, D, device="cuda") * 0.2).bfloat16()
    h, t = data(mk(0))
    d = torch.full((T,), 1 / T, device="cuda")
    dw = torch.zeros(V, D, device="cuda")
    out = torch.empty(V, D, device="cuda", dtype=B)

    def run():
        dw.zero_()
        loss, dh, _ = moe.linear_cross_entropy_step(h, w, t, d, dweight=dw)
        norm = moe.clip_grads([dw], 0.01, out=[out])
        return loss, dh, norm

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run()
    for seed in (1, 2):
        for a, b in zip((h, t), data(mk(seed))):
            a.copy_(b)
        graph.replay()
        kept = [x.clone() for x in (*got, out)]
        want = (*run(), out)
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_two_streams_at_once():
    """Two calls under way together, each with its own workspace."""
    h = torch.randn(300, 128, device="cuda").bfloat16()
    w = torch.randn(5000, 128, device="cuda").bfloat16() * 0.1
    t = torch.randint(5000, (300,), device="cuda")
    d = torch.rand(300, device="cuda")
    want = [moe.linear_cross_entropy_step(h[:n], w, t[:n], d[:n]) for n in (300, 100)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i, n in enumerate((300, 100)):
            with torch.cuda.stream(streams[i]):
                got[i].append(moe.linear_cross_entropy_step(h[:n], w, t[:n], d[:n]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))


def test_head_refuses_another_shape():
    with pytest.raises(ValueError):
        moe.LMHead(100, 64, weight=torch.nn.Parameter(torch.zeros(64, 100, device="cuda")))


def test_example():
    spec = importlib.util.spec_from_file_location("next_token", os.path.join(ROOT, "examples", "next_token_training.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, norms = mod.train(steps=2, tokens=96, vocabulary=500)
    assert len(losses) == len(norms) == 2 and all(x == x and 0 < x < 1e4 for x in losses + norms)
