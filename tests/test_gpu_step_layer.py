"""The operators around the layer under autograd, and the example that runs
them with the layer."""
import importlib.util
import os

import pytest
import torch

import top_routed_grouped_gb300 as moe
import top_routed_grouped_gb300.step_layer  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def plain_norm(v, w):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w


def close(a, b, what):
    """FP32 through a few chained operators: 2^-24 of the result's norm times
    the roundings on the way (some hundreds)."""
    a, b = a.double(), b.double()
    assert float((a - b).norm()) <= 2e-5 * float(b.norm()) + 1e-12, what


@pytest.mark.parametrize("gate", [None, "token", "channel", "element"])
@pytest.mark.parametrize("post", [True, False])
def test_gradients_through_a_chain(gate, post):
    """embedding -> norm -> join -> logits -> distillation, against torch's
    autograd over the same formulas in float64."""
    T, V, H, K = 37, 90, 64, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(V, (T,), generator=g, device="cuda")
    t_ids = torch.randint(V, (T, K), generator=g, device="cuda").int()
    t_logits, weight = rn(T, K), rn(T)
    p = {"table": 0.3 * rn(V, H), "w1": 1 + 0.1 * rn(H), "w_post": 1 + 0.1 * rn(H), "w_pre": 1 + 0.1 * rn(H),
         "mix": 0.2 * rn(H, H)}
    if gate:
        p["gate"] = {"token": rn(T, 1), "channel": rn(H), "element": rn(T, H)}[gate]
    if not post:
        del p["w_post"]
    a = {k: v.clone().requires_grad_() for k, v in p.items()}
    b = {k: v.double().requires_grad_() for k, v in p.items()}

    r = moe.step_layer.EmbedFunction.apply(a["table"], ids, 2.0, None, None)
    h = moe.step_layer.BlockNormFunction.apply(r, None, None, a["w1"], None, 1.0, 1e-6, 0.0, None)
    r, h = moe.step_layer.BlockNormFunction.apply(r, torch.tanh(h @ a["mix"]), a.get("w_post"), a["w_pre"],
                                                  a.get("gate"), 0.5, 1e-6, 0.0, None)
    loss = moe.distillation_loss(h @ a["table"].t() + r.sum(1, keepdim=True) * 0, t_ids, t_logits, 2.0, 4.0)
    (loss @ weight + r.square().sum() * 0.01).backward()

    r = b["table"][ids] * 2.0
    h = plain_norm(r, b["w1"])
    y = torch.tanh(h @ b["mix"])
    y = plain_norm(y, b["w_post"]) if post else y
    r = r + 0.5 * (b["gate"] if gate else 1.0) * y
    h = plain_norm(r, b["w_pre"])
    z = h @ b["table"].t() / 2.0
    q = torch.softmax(t_logits.double() / 2.0, 1)
    want = 4.0 * (q * (q.log() - torch.log_softmax(z, 1).gather(1, t_ids.long()))).sum(1)
    (want @ weight.double() + r.square().sum() * 0.01).backward()

    close(loss, want, "loss")
    for k in a:
        close(a[k].grad, b[k].grad, k)


def test_outputs_without_gradient():
    """Only one of r_out and h is used, or neither norm is there."""
    T, H = 9, 32
    r, y, w = (torch.randn(s, device="cuda", requires_grad=True) for s in ((T, H), (T, H), (H,)))
    for use in (0, 1):
        out = moe.step_layer.BlockNormFunction.apply(r, y, w, w, None, 1.0, 1e-6, 0.0, None)
        got = torch.autograd.grad(out[use].sum(), (r, y, w))
        rd, yd, wd = (t.detach().double().requires_grad_() for t in (r, y, w))
        s = rd + plain_norm(yd, wd)
        want = torch.autograd.grad((s, plain_norm(s, wd))[use].sum(), (rd, yd, wd))
        for a, b, n in zip(got, want, "ryw"):
            assert float((a.double() - b).abs().max()) <= 1e-5 * (1 + float(b.abs().max())), n
    alone = moe.BlockNorm(H, post=False, pre=False, scale=0.5, dtype=torch.float32)
    out = alone(r, y)
    assert torch.allclose(out, r + 0.5 * y)
    gr, gy = torch.autograd.grad(out.sum(), (r, y))
    assert torch.equal(gr, torch.ones_like(r)) and torch.equal(gy, torch.full_like(y, 0.5))


def test_values_that_autograd_saved_are_not_overwritten_unseen():
    """A product saves its factors; a call then writes over one of them."""
    r, y, w = (torch.randn(s, device="cuda") for s in ((6, 16), (6, 16), (16,)))
    z, t_ids, t = torch.randn(6, 16, device="cuda"), torch.zeros(6, 1, dtype=torch.int32, device="cuda"), torch.ones(6, 1, device="cuda")
    one, lse = torch.ones(6, device="cuda"), torch.logsumexp(z, 1)
    for x, write in ((r, lambda x: moe.block_norm(x, y, None, w, inplace=True)),
                     (torch.zeros(9, 16, device="cuda"), lambda x: moe.embed_backward(t_ids[:, 0], y, 9, dtable=x)),
                     (z, lambda x: moe.distill_step(x, t_ids, t, one, out=x)),
                     (z, lambda x: moe.distill_backward(one, lse, x, t_ids, t, out=x)),
                     (z[:, :9], lambda x: moe.distill_step(x, t_ids, t, one, out=x))):
        k = torch.ones_like(x).requires_grad_()
        out = k * x
        write(x)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.sum().backward()
    with torch.inference_mode():
        x = torch.randn(6, 16, device="cuda")
        assert moe.block_norm(x, y, None, w, inplace=True)[0] is x


def test_modules():
    emb = moe.TokenEmbedding(50, 64, scale=8.0, padding_id=3, dtype=torch.bfloat16, out_dtype=torch.float32)
    ids = torch.tensor([3, 7, 7, 49], device="cuda")
    out = emb(ids)
    assert out.dtype == torch.float32 and out.shape == (4, 64)
    out.sum().backward()
    grad = emb.weight.grad
    assert grad.dtype == torch.bfloat16 and not grad[3].any() and (grad[7] == 16).all() and (grad[49] == 8).all()
    norm = moe.BlockNorm(64, weight_offset=1.0)
    assert not norm.w_post.any() and not norm.w_pre.any()
    r_out, h = norm(out.detach(), torch.ones(4, 64, device="cuda", dtype=torch.bfloat16))
    assert r_out.dtype == torch.float32 and h.dtype == torch.bfloat16


def test_the_last_token_as_padding():
    emb = moe.TokenEmbedding(50, 8, padding_id=-1, dtype=torch.float32)
    emb(torch.tensor([49, 7, 49], device="cuda")).sum().backward()
    assert not emb.weight.grad[49].any() and (emb.weight.grad[7] == 1).all()


def test_example_learns():
    spec = importlib.util.spec_from_file_location("distill_training", os.path.join(ROOT, "examples", "distill_training.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(steps=12)
    assert all(v == v for v in losses) and losses[-1] < 0.7 * losses[0], losses
    assert moe.moe_device_status(reset=True) == 0


def test_step_under_graph_capture():
    """The operators replay from a CUDA graph on new values, bit for bit."""
    T, V, H, K = 64, 4096, 256, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    table = torch.randn(V, H, generator=g, device="cuda").bfloat16()
    y = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = torch.ones(H, device="cuda").bfloat16()
    z = torch.randn(T, V, generator=g, device="cuda").bfloat16()
    ids = torch.randint(V, (T,), generator=g, device="cuda")
    t_ids = torch.randint(V, (T, K), generator=g, device="cuda").int()
    t_logits, weight = torch.randn(T, K, generator=g, device="cuda"), torch.ones(T, device="cuda")

    def step():
        r = moe.embed(table, ids, out_dtype=torch.float32)
        r_out, h = moe.block_norm(r, y, w, w)
        d = moe.block_norm_backward(r, h, r_out, y, w, w)
        loss, dz = moe.distill_step(z, t_ids, t_logits, weight)
        return [r_out, h, d["dr"], d["dy"], d["dw_pre"], d["dw_post"], loss, dz, moe.embed_backward(ids, d["dr"], V)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (3, 4):
        g.manual_seed(seed)
        ids.copy_(torch.randint(V, (T,), generator=g, device="cuda"))
        z.copy_(torch.randn(T, V, generator=g, device="cuda"))
        y.copy_(torch.randn(T, H, generator=g, device="cuda"))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
