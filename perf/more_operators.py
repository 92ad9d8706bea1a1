"""The end of a training step, as cases to be measured: the loss of the next
token from hidden rows, and the gradients' global norm with clipping.

``ce_fwd`` / ``ce_bwd`` / ``ce_step``
    ``linear_cross_entropy``: logits of the output embedding and their softmax
    cross entropy, without the logits as an operand or a result.  With
    x_t = scale * weight @ hidden_t over the vocabulary,
        lse_t  = log sum_v exp(x_tv)
        loss_t = lse_t - x_t[target_t] + z_loss * lse_t^2
        dx_tv  = dloss_t * ((1 + 2 z_loss lse_t) exp(x_tv - lse_t) - [v = target_t])
        dhidden = scale * dx @ weight,  dweight = scale * dx^T @ hidden
    A row whose target is IGNORE (prompts, padding) has loss and lse 0 and no
    part in the gradients.  The step gives loss and gradients in one call, for
    a dloss that is known beforehand.
``norm`` / ``clip``
    ``grad_norm``: the 2-norm over all elements of many tensors.
    ``clip_grads``: that norm, and every tensor times
    min(1, max_norm / (norm + EPS)), written to other tensors here (float32
    gradients as they were accumulated, handed on in the parameters' type).
"""
import math
import random

import torch

own = False

IGNORE = -100
EPS = 1e-6


def _dt(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _size(name):
    return {"bf16": 2, "f32": 4}[name]


# ------------------------------------------------------------------- the cases
def listed():
    ce = dict(dtype="bf16", masked=False, scale=1.0, z_loss=0.0)
    return [
        # Scoring the last few tokens of a prompt: one pass over the table, where latency counts.
        dict(ce, name="ce fwd few rows", op="ce_fwd", T=5, D=2048, V=32000),
        # Perplexity of a held-out batch at an odd vocabulary.
        dict(ce, name="ce fwd odd vocabulary", op="ce_fwd", T=4096, D=2048, V=50257),
        # The gradient by itself, from the forward's lse; half of the rows are prompts; sizes that fit no tile.
        dict(ce, name="ce bwd ragged", op="ce_bwd", T=2049, D=1000, V=32001, masked=True),
        # A small float32 model, as its tests run it.
        dict(ce, name="ce step f32 small", op="ce_step", T=333, D=256, V=5003, dtype="f32", z_loss=1e-3),
        # A micro-batch of a large vocabulary, where reading and writing the tables counts.
        dict(ce, name="ce step micro batch", op="ce_step", T=256, D=2048, V=131072),
        # Instruction tuning: half of the rows are prompts; z loss, scaled logits.
        dict(ce, name="ce step masked", op="ce_step", T=8192, D=4096, V=32000, masked=True, scale=0.5, z_loss=1e-4),
        # The step of a full 8K batch over a large vocabulary.
        dict(ce, name="ce step 8K", op="ce_step", T=8192, D=2048, V=131072),
        # Monitoring of a small model: some dozens of tensors, where only latency counts.
        dict(name="norm small model", op="norm", n=34, numel=9_500_000, dtype="f32", odtype="f32", max_norm=1.0),
        # Many tensors of very different sizes in bfloat16 (norm weights among matrices), at odd offsets.
        dict(name="clip many tensors", op="clip", n=1500, numel=300_000_000, dtype="bf16", odtype="bf16", max_norm=1.0),
        # A few tensors that stay on chip between the norm and the scaling.
        dict(name="clip small model", op="clip", n=34, numel=9_500_001, dtype="f32", odtype="bf16", max_norm=1.0),
        # The float32 gradients of an MoE layer of 512 experts, clipped and handed on in its weights' type.
        dict(name="clip layer", op="clip", n=6, numel=1_620_000_000, dtype="f32", odtype="bf16", max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a multiple of 64 mostly, any number otherwise."""
    n = _log_int(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(["ce_fwd", "ce_bwd", "ce_step", "norm", "clip"])
    if op.startswith("ce"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        most = 1 << (39 if dtype == "bf16" else 33)  # T * D * V
        D = _width(rng, 64, 4096 if dtype == "bf16" else 1024)
        V = _width(rng, 1000, min(131072, most // D // 64))
        T = _log_int(rng, 1, min(16384, most // D // V))
        return dict(op=op, T=T, D=D, V=V, dtype=dtype, masked=T > 8 and rng.random() < 0.4,
                    scale=rng.choice([1.0, 1.0, 0.25]), z_loss=rng.choice([0.0, 1e-4]))
    numel = _log_int(rng, 10_000, 1_000_000_000)
    dtype = rng.choice(["bf16", "f32"])
    return dict(op=op, n=_log_int(rng, 1, min(2000, max(2, numel // 100))), numel=numel, dtype=dtype,
                odtype=rng.choice([dtype, "bf16"]), max_norm=rng.choice([1.0, 1e9]))


def _sizes(case):
    """Sizes of ``n`` tensors, about ``numel`` elements in all: a few hold most of them."""
    n, total = case["n"], case["numel"]
    rng = random.Random(1000003 * n + total)
    share = [math.exp(rng.gauss(0.0, 2.0)) for _ in range(n)]
    all_of = sum(share)
    return [max(1, int(total * x / all_of)) for x in share]


# ------------------------------------------------------------------ their inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"].startswith("ce"):
        T, D, V, dt = case["T"], case["D"], case["V"], _dt(case["dtype"])
        w = torch.randn(V, D, generator=g, device="cuda").mul_(2.0 / math.sqrt(D))
        # Frequencies of text: the token of rank n comes about 1/n of the time.
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(V)) - 1.0).long().clamp_(0, V - 1)
        # Normed rows of a model that has learned something: the target's logit lies above the others.
        h = torch.randn(T, D, generator=g, device="cuda")
        h += (1.0 + torch.rand(T, 1, generator=g, device="cuda")) / case["scale"] * w[ids]
        if case["masked"]:
            ids[torch.rand(T, generator=g, device="cuda").argsort()[:T // 2]] = IGNORE
        s["hidden"], s["weight"], s["targets"] = h.to(dt), w.to(dt), ids
        if case["op"] != "ce_fwd":
            s["dloss"] = (0.5 + torch.rand(T, generator=g, device="cuda")) / T  # the batch's mean, tokens weighted
        if case["op"] == "ce_bwd":
            lse = torch.cat([torch.logsumexp(s["hidden"][t:t + 1024].float() @ s["weight"].float().t() * case["scale"], 1)
                             for t in range(0, T, 1024)])
            s["lse"] = torch.where(ids == IGNORE, 0.0, lse)
        return s
    sizes = _sizes(case)
    total = sum(sizes)
    flat = torch.empty(total, device="cuda", dtype=_dt(case["dtype"]))
    for a in range(0, total, 1 << 27):
        b = min(total, a + (1 << 27))
        flat[a:b] = torch.randn(b - a, generator=g, device="cuda").mul_(1e-3)
    s["flat"], s["grads"] = flat, list(flat.split(sizes))
    if case["op"] == "clip":
        s["out"] = torch.empty(total, device="cuda", dtype=_dt(case["odtype"]))
        s["outs"] = list(s["out"].split(sizes))
    return s


# --------------------------------------------------------------- the plain forms
def _plain_ce(s):
    keep = s["targets"] != IGNORE
    ids = torch.where(keep, s["targets"], 0)
    h, w = s["hidden"].float() * keep[:, None], s["weight"].float()
    x = h @ w.t()
    if s["scale"] != 1.0:
        x *= s["scale"]
    loss, out = None, []
    if s["op"] == "ce_bwd":
        lse = s["lse"]
    else:
        m = x.amax(1, keepdim=True)
        lse = (x - m).exp_().sum(1).log_() + m[:, 0]
        lse = torch.where(keep, lse, 0.0)
        loss = lse - x.gather(1, ids[:, None])[:, 0] + s["z_loss"] * lse * lse
        out.append(torch.where(keep, loss, 0.0))
    if s["op"] == "ce_fwd":
        return out[0], lse
    d = torch.where(keep, s["dloss"], 0.0)
    x = x.sub_(lse[:, None]).exp_()
    x *= (d * (1.0 + 2.0 * s["z_loss"] * lse))[:, None]
    x[torch.arange(x.shape[0], device=x.device), ids] -= d
    if s["scale"] != 1.0:
        x *= s["scale"]
    return tuple(out) + ((x @ w).to(s["hidden"].dtype), (x.t() @ h).to(s["weight"].dtype))


def _plain_norm(s):
    squares = []
    for t in s["grads"]:
        part = torch.zeros((), device=t.device, dtype=torch.float64)
        for a in range(0, t.numel(), 1 << 24):
            part += t[a:a + (1 << 24)].float().square().sum(dtype=torch.float64)
        squares.append(part)
    return torch.stack(squares).sum().sqrt().float()


def _plain_clip(s):
    norm = _plain_norm(s)
    c = (s["max_norm"] / (norm + EPS)).clamp(max=1.0)
    for t, o in zip(s["grads"], s["outs"]):
        o.copy_(t.float() * c)
    return norm, s["out"]


# ------------------------------------------------------------------ one pass each
def run(s):
    op = s["op"]
    if not own:
        return _plain_ce(s) if op.startswith("ce") else _plain_norm(s) if op == "norm" else _plain_clip(s)
    import top_routed_grouped_gb300 as moe

    if op == "norm":
        return moe.grad_norm(s["grads"])
    if op == "clip":
        return moe.clip_grads(s["grads"], s["max_norm"], eps=EPS, out=s["outs"]), s["out"]
    kw = dict(scale=s["scale"], z_loss=s["z_loss"], ignore_index=IGNORE)
    if op == "ce_fwd":
        return moe.linear_cross_entropy(s["hidden"], s["weight"], s["targets"], **kw)
    if op == "ce_bwd":
        return moe.linear_cross_entropy_backward(s["dloss"], s["lse"], s["hidden"], s["weight"], s["targets"], **kw)
    return moe.linear_cross_entropy_step(s["hidden"], s["weight"], s["targets"], s["dloss"], **kw)


# ---------------------------------------------------------------- what it has to do
def work(case):
    if case["op"].startswith("ce"):
        T, D, V, e = case["T"], case["D"], case["V"], _size(case["dtype"])
        rows = T - T // 2 if case["masked"] else T  # (those that have a target)
        tables = (rows * D + V * D) * e
        if case["op"] == "ce_fwd":
            return {"bytes": tables + 8 * T + 8 * T, "flops": 2 * rows * D * V}
        outputs = (T * D + V * D) * e
        # The logits once, and both gradients from them.
        return {"bytes": tables + outputs + 8 * T + 8 * T, "flops": 6 * rows * D * V}
    n = sum(_sizes(case))
    if case["op"] == "norm":
        return {"bytes": n * _size(case["dtype"]) + 4, "flops": 2 * n}
    return {"bytes": n * (_size(case["dtype"]) + _size(case["odtype"])) + 4, "flops": 3 * n}


# ------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    if case["op"].startswith("ce"):
        if case["T"] * case["D"] * case["V"] > 1.0e12:
            return None  # minutes in 64 bits
        s = prepare(case, seed)
        w = s["weight"].double()
        T, scale, z = case["T"], case["scale"], case["z_loss"]
        bwd = case["op"] != "ce_fwd"
        loss = torch.zeros(T, dtype=torch.float64, device="cuda")
        lses = torch.zeros(T, dtype=torch.float64, device="cuda")
        dh = torch.zeros(T, case["D"], dtype=torch.float64, device="cuda") if bwd else None
        dw = torch.zeros_like(w) if bwd else None
        rows = torch.nonzero(s["targets"] >= 0)[:, 0]
        step = max(1, (1 << 27) // case["V"])
        for r in rows.split(step):
            h, t = s["hidden"][r].double(), s["targets"][r]
            x = torch.einsum("td,vd->tv", h, w) * scale
            lse = torch.logsumexp(x, dim=1)
            loss[r] = lse - x[torch.arange(len(r), device="cuda"), t] + z * lse ** 2
            lses[r] = lse
            if bwd:
                if case["op"] == "ce_bwd":
                    lse = s["lse"][r].double()
                u = s["dloss"][r].double()
                p = torch.exp(x - lse[:, None]) * (u * (1 + 2 * z * lse))[:, None]
                p.scatter_add_(1, t[:, None], -u[:, None])
                dh[r] = scale * torch.einsum("tv,vd->td", p, w)
                dw += scale * torch.einsum("tv,td->vd", p, h)
        return (loss, lses) if not bwd else (dh, dw) if case["op"] == "ce_bwd" else (loss, dh, dw)
    s = prepare(case, seed)
    flat, total = s["flat"], 0.0
    for part in flat.split(1 << 26):
        v = part.double()
        total += float(torch.dot(v, v))
    norm = math.sqrt(total)
    if case["op"] == "norm":
        return torch.tensor(norm, dtype=torch.float64)
    c = min(1.0, case["max_norm"] / (norm + EPS))
    out = torch.empty(flat.numel(), dtype=torch.float64, device="cuda")
    for a in range(0, flat.numel(), 1 << 26):
        out[a:a + (1 << 26)] = flat[a:a + (1 << 26)].double() * c
    return torch.tensor(norm, dtype=torch.float64), out
