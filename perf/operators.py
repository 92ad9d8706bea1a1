"""The operators of a training step around the MoE layer, as cases to be measured.

Three operators, each in its directions:

``norm_fwd`` / ``norm_bwd``
    ``block_norm``: the norm after a block, its gate, the scaled residual sum
    and the norm before the next block, in one pass over the rows, and its
    gradients.  With n(v; w) = v / sqrt(mean(v^2) + eps) * (w + offset):
        r' = r + scale * gate * n(y; w_post)        h = n(r'; w_pre)
    ``post`` false: y enters as it is; ``pre`` false: no h; ``block`` false: no
    y at all (h = n(r; w_pre)).  ``gate``: none, one number a token, one a
    channel, or one an element.
``embed_fwd`` / ``embed_bwd``
    ``embed``: out[t] = scale * table[id_t]; its gradient sums, for every row
    of the table, the rows of ``dout`` whose token it is.
``distill_fwd`` / ``distill_bwd`` / ``distill_step``
    ``distill``: the cross entropy gap between a teacher, known by the logits
    of its K likeliest tokens, and the student's full softmax q:
        p = softmax(teacher / tau) over the K kept,  q = softmax(student / tau)
        loss_t = scale * sum_k p_k (log p_k - log q_{id_k})
        dlogits_t = weight_t * scale / tau * (q - p scattered to its ids)
    An id of -1 is a slot that is not there; a row without slots has no loss
    and no gradient.  The step computes loss and gradient in one call.
"""
import math

import torch

own = False

EPS = 1e-6


def _dt(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _size(name):
    return {"bf16": 2, "f32": 4}[name]


# ------------------------------------------------------------------- the cases
def listed():
    norm = dict(post=True, pre=True, block=True, gate="none", dtype="bf16", rdtype="bf16", offset=0.0, scale=1.0)
    return [
        # One decoding step of eight sequences: the join between two blocks, where only latency counts.
        dict(norm, name="norm fwd decode", op="norm_fwd", T=8, H=2048, gate="token"),
        # A packed 8K sequence at the layer's hidden size, the residual stream kept in 32 bits.
        dict(norm, name="norm fwd 8K", op="norm_fwd", T=8192, H=2048, rdtype="f32", scale=0.5),
        # A narrow float32 model with an odd hidden size and a gate for each channel.
        dict(norm, name="norm bwd f32 odd", op="norm_bwd", T=4099, H=1001, gate="channel", dtype="f32", rdtype="f32"),
        # The backward of a large batch, gated element by element, norms that store w - 1.
        dict(norm, name="norm bwd 32K", op="norm_bwd", T=32768, H=2048, gate="element", offset=1.0),
        # Embedding of a prompt chunk, scaled by sqrt(H), from a table that L2 does not hold.
        dict(name="embed fwd 16K", op="embed_fwd", T=16384, H=2048, V=131072, dtype="bf16", odtype="bf16", padding=False),
        # One token for each of sixteen sequences.
        dict(name="embed fwd decode", op="embed_fwd", T=16, H=2048, V=131072, dtype="bf16", odtype="f32", padding=False),
        # The gradient of a small vocabulary's table: long runs of equal tokens, with a padding token.
        dict(name="embed bwd 4K", op="embed_bwd", T=4096, H=2048, V=32000, dtype="bf16", odtype="f32", padding=True),
        # The gradient of a large table from a large batch.
        dict(name="embed bwd 64K", op="embed_bwd", T=65536, H=2048, V=131072, dtype="bf16", odtype="bf16", padding=False),
        # Monitoring of a held-out batch: the loss alone, at an odd vocabulary in float32.
        dict(name="distill fwd odd", op="distill_fwd", T=333, V=50257, K=8, dtype="f32", tau=1.0, empty=0),
        # The gradient by itself, from the forward's saved statistics, prompts masked out.
        dict(name="distill bwd 4K", op="distill_bwd", T=4096, V=32000, K=32, dtype="bf16", tau=2.0, empty=1),
        # A micro-batch of a few rows: the step in one call.
        dict(name="distill step few rows", op="distill_step", T=16, V=131072, K=64, dtype="bf16", tau=1.0, empty=0),
        # The step of a full 8K batch over a large vocabulary.
        dict(name="distill step 8K", op="distill_step", T=8192, V=131072, K=64, dtype="bf16", tau=2.0, empty=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a multiple of 64 mostly, any number otherwise."""
    n = _log_int(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "embed_fwd", "embed_bwd", "distill_fwd", "distill_bwd", "distill_step"])
    if op.startswith("norm"):
        H = _width(rng, 64, 8192)
        T = _log_int(rng, 1, min(65536, (1 << 26) // H))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        block = op == "norm_bwd" or rng.random() < 0.8
        post, pre = rng.choice([(True, True), (False, True), (True, False)]) if block else (False, True)
        return dict(op=op, T=T, H=H, post=post, pre=pre, block=block,
                    gate=rng.choice(["none", "token", "channel", "element"]) if block else "none",
                    dtype=dtype, rdtype=rng.choice([dtype, "f32"]), offset=rng.choice([0.0, 1.0]),
                    scale=rng.choice([1.0, 0.5]))
    if op.startswith("embed"):
        H = _width(rng, 64, 8192)
        V = _log_int(rng, 1000, min(262144, (1 << 28) // H))
        T = _log_int(rng, 1, min(65536, (1 << 27) // H))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, T=T, H=H, V=V, dtype=dtype, odtype=rng.choice([dtype, "f32"]), padding=rng.random() < 0.3)
    V = _width(rng, 1000, 262144)
    T = _log_int(rng, 1, min(16384, (1 << 28) // V))
    return dict(op=op, T=T, V=V, K=_log_int(rng, 1, 256), dtype=rng.choice(["bf16", "bf16", "f32"]),
                tau=rng.choice([1.0, 2.0, 0.7]), empty=rng.choice([0, 1]))


def _empty_rows(case):
    """Rows whose teacher has no slot (prompts): an eighth of the batch, or none."""
    return case["T"] // 8 if case["empty"] else 0


# ------------------------------------------------------------------ their inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32, mul=1.0, add=0.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(mul).add_(add).to(dtype)

    s = dict(case)
    op, T = case["op"], case["T"]
    if op.startswith("norm"):
        H, dt, rdt = case["H"], _dt(case["dtype"]), _dt(case["rdtype"])
        base = 1.0 - case["offset"]  # a norm that stores w - 1 has weights near 0
        s["r"] = randn(T, H, dtype=rdt, mul=2.0)
        s["y"] = randn(T, H, dtype=dt, mul=0.3) if case["block"] else None
        s["w_post"] = randn(H, dtype=dt, mul=0.1, add=base) if case["post"] else None
        s["w_pre"] = randn(H, dtype=dt, mul=0.1, add=base) if case["pre"] else None
        s["g"] = {"none": lambda: None, "token": lambda: torch.sigmoid(randn(T, 1)),
                  "channel": lambda: randn(H, dtype=dt, mul=0.1, add=0.5),
                  "element": lambda: torch.sigmoid(randn(T, H)).to(dt)}[case["gate"]]()
        if op == "norm_bwd":  # s["r"] is the stored r' of the forward
            s["dr_out"] = randn(T, H, dtype=rdt)
            s["dh"] = randn(T, H, dtype=dt) if case["pre"] else None
    elif op.startswith("embed"):
        V, H = case["V"], case["H"]
        # Frequencies of text: the token of rank n comes about 1/n of the time.
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        s["ids"] = (torch.exp(u * math.log(V)) - 1.0).long().clamp_(0, V - 1)
        s["scale"] = math.sqrt(H)
        s["padding_id"] = 0 if case["padding"] else None
        if op == "embed_fwd":
            s["table"] = randn(V, H, dtype=_dt(case["dtype"]), mul=0.02)
        else:
            s["dout"] = randn(T, H, dtype=_dt(case["odtype"]))
    else:
        V, K = case["V"], case["K"]
        z = torch.empty(T, V, device="cuda", dtype=_dt(case["dtype"]))
        for t in range(0, T, 1024):
            z[t:t + 1024] = randn(min(1024, T - t), V, mul=2.0).to(z.dtype)
        # K different ids a row, in no order; a student that has learned some of its teacher.
        part = V // K
        ids = torch.arange(K, device="cuda") * part + torch.randint(part, (T, K), generator=g, device="cuda")
        ids = ids.gather(1, torch.rand(T, K, generator=g, device="cuda").argsort(1))
        t_logits = randn(T, K, mul=2.0, add=6.0).sort(1, descending=True).values
        z.scatter_(1, ids, (0.7 * t_logits + randn(T, K)).to(z.dtype))
        if case["empty"]:  # lists of different lengths, and rows without any
            keep = torch.randint(1, K + 1, (T, 1), generator=g, device="cuda")
            ids = torch.where(torch.arange(K, device="cuda") < keep, ids, -1)
            ids[torch.randperm(T, generator=g, device="cuda")[:_empty_rows(case)]] = -1
        s["z"], s["ids"], s["t_logits"] = z, ids.to(torch.int32), t_logits
        s["weight"] = torch.rand(T, generator=g, device="cuda") / T  # the batch's mean, tokens weighted
        if op == "distill_bwd":
            s["lse"] = torch.cat([torch.logsumexp(z[t:t + 1024].float() / case["tau"], 1) for t in range(0, T, 1024)])
    return s


# --------------------------------------------------------------- the plain forms
def _plain_norm_fwd(s):
    r, o = s["r"].float(), s["offset"]
    if s["y"] is not None:
        n = s["y"].float()
        if s["post"]:
            n = n * torch.rsqrt((n * n).mean(1, keepdim=True) + EPS) * (s["w_post"].float() + o)
        if s["g"] is not None:
            n = n * s["g"].float()
        r = r + s["scale"] * n
    out = [r.to(s["r"].dtype)] if s["y"] is not None else []
    if s["pre"]:
        h = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * (s["w_pre"].float() + o)
        out.append(h.to(_dt(s["dtype"])))
    return out


def _plain_norm_bwd(s):
    o, out = s["offset"], {}
    d = s["dr_out"].float()
    if s["pre"]:
        r, dh = s["r"].float(), s["dh"].float()
        rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
        xhat, dx = r * rstd, dh * (s["w_pre"].float() + o)
        out["dw_pre"] = (dh * xhat).sum(0)
        d = d + rstd * (dx - xhat * (dx * xhat).mean(1, keepdim=True))
    out["dr"] = d.to(s["r"].dtype)
    y, dn = s["y"].float(), s["scale"] * d
    if s["post"]:
        rstd = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        xhat, w = y * rstd, s["w_post"].float() + o
        n = xhat * w
    else:
        n = y
    if s["g"] is not None:
        dg = dn * n
        if s["gate"] == "element":
            out["dgate"] = dg.to(s["g"].dtype)
        else:
            out["dgate"] = dg.sum(0) if s["gate"] == "channel" else dg.sum(1, keepdim=True)
        dn = dn * s["g"].float()
    if s["post"]:
        out["dw_post"] = (dn * xhat).sum(0)
        dx = dn * w
        dn = rstd * (dx - xhat * (dx * xhat).mean(1, keepdim=True))
    out["dy"] = dn.to(s["y"].dtype)
    return out


def _plain_embed_fwd(s):
    return (s["table"][s["ids"]].float() * s["scale"]).to(_dt(s["odtype"]))


def _plain_embed_bwd(s):
    d = s["dout"].float() * s["scale"]
    if s["padding_id"] is not None:
        d = d * (s["ids"] != s["padding_id"]).unsqueeze(1)
    return torch.zeros(s["V"], s["H"], device=d.device).index_add_(0, s["ids"], d)


def _teacher(s):
    """p over the K slots, log p, and the slots' ids (0 where there is none)."""
    there = s["ids"] >= 0
    t = torch.where(there, s["t_logits"] / s["tau"], -math.inf)
    m = t.amax(1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    e = torch.exp(t - m)
    total = e.sum(1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    return p, torch.where(there, t - m - torch.log(total), 0.0), s["ids"].clamp_min(0).long()


def _plain_distill_loss(s):
    z = s["z"].float() / s["tau"]
    m = z.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    p, log_p, ids = _teacher(s)
    loss = (p * (log_p - (z.gather(1, ids) - lse))).sum(1)
    return loss, lse.squeeze(1), z, p, ids


def _plain_distill_grad(s, z, lse, p, ids, weight):
    d = torch.exp(z - lse.unsqueeze(1)) * p.sum(1, keepdim=True)
    d.scatter_add_(1, ids, -p)
    return (d * (weight / s["tau"]).unsqueeze(1)).to(s["z"].dtype)


def _plain(s):
    op = s["op"]
    if op == "norm_fwd":
        return _plain_norm_fwd(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "embed_fwd":
        return _plain_embed_fwd(s)
    if op == "embed_bwd":
        return _plain_embed_bwd(s)
    if op == "distill_bwd":
        p, _, ids = _teacher(s)
        return _plain_distill_grad(s, s["z"].float() / s["tau"], s["lse"], p, ids, s["weight"])
    loss, lse, z, p, ids = _plain_distill_loss(s)
    if op == "distill_fwd":
        return loss, lse
    return loss, _plain_distill_grad(s, z, lse, p, ids, s["weight"])


# --------------------------------------------------------- the framework's calls
def _own(s):
    import top_routed_grouped_gb300 as moe

    op = s["op"]
    if op == "norm_fwd":
        r_out, h = moe.block_norm(s["r"], s["y"], s["w_post"], s["w_pre"], gate=s["g"], scale=s["scale"], eps=EPS,
                                  weight_offset=s["offset"], dtype=_dt(s["dtype"]))
        return [x for x in (r_out if s["y"] is not None else None, h) if x is not None]
    if op == "norm_bwd":
        d = moe.block_norm_backward(s["dr_out"], s["dh"], s["r"], s["y"], s["w_post"], s["w_pre"], gate=s["g"],
                                    scale=s["scale"], eps=EPS, weight_offset=s["offset"])
        return {k: v for k, v in d.items() if v is not None}
    if op == "embed_fwd":
        return moe.embed(s["table"], s["ids"], scale=s["scale"], out_dtype=_dt(s["odtype"]))
    if op == "embed_bwd":
        return moe.embed_backward(s["ids"], s["dout"], s["V"], scale=s["scale"], padding_id=s["padding_id"])
    if op == "distill_fwd":
        return moe.distill(s["z"], s["ids"], s["t_logits"], temperature=s["tau"])
    if op == "distill_bwd":
        return moe.distill_backward(s["weight"], s["lse"], s["z"], s["ids"], s["t_logits"], temperature=s["tau"])
    return moe.distill_step(s["z"], s["ids"], s["t_logits"], s["weight"], temperature=s["tau"])


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- their work
def work(case):
    op, T = case["op"], case["T"]
    if op.startswith("norm"):
        H, e, r = case["H"], _size(case["dtype"]), _size(case["rdtype"])
        gate = {"none": 0, "token": 4 * T, "channel": e * H, "element": e * T * H}[case["gate"]]
        weights = e * H * (case["post"] + case["pre"])
        if op == "norm_fwd":  # r, y, gate in; r', h out
            n = T * H * (r + (e + r) * case["block"] + e * case["pre"]) + gate + weights
            return {"bytes": n, "flops": T * H * (4 * case["pre"] + 4 * case["post"] + 3 * case["block"])}
        # dr', y in and dy out; with a norm before the next block also r' and dh in and dr out (without one dr is dr');
        # the gradients of what is learned in float32
        n = T * H * (r + 2 * e + (2 * r + e) * case["pre"]) + H * (e + 4) * (case["post"] + case["pre"])
        n += gate + {"none": 0, "token": 4 * T, "channel": 4 * H, "element": e * T * H}[case["gate"]]
        return {"bytes": n, "flops": T * H * (10 * case["pre"] + 10 * case["post"] + 4)}
    if op.startswith("embed"):
        H, V = case["H"], case["V"]
        if op == "embed_fwd":  # the different rows of the table among T draws with frequencies 1/n: rank n is drawn with log((n + 1) / n) / log(V)
            seen = _seen(T, V)
            return {"bytes": seen * H * _size(case["dtype"]) + T * H * _size(case["odtype"]) + 8 * T, "flops": T * H}
        return {"bytes": T * H * _size(case["odtype"]) + 4 * V * H + 8 * T, "flops": 2 * T * H}
    V, K, e = case["V"], case["K"], _size(case["dtype"])
    read = (T - _empty_rows(case)) * V * e + 8 * T * K
    if op == "distill_fwd":
        return {"bytes": read + 8 * T, "flops": 4 * T * V}
    return {"bytes": read + T * V * e + 8 * T, "flops": (4 if op == "distill_bwd" else 8) * T * V}


def _seen(T, V):
    """How many different tokens T draws are expected to hold."""
    n = torch.arange(1, V + 1, dtype=torch.float64)
    return float((1 - torch.exp(T * torch.log1p(-torch.log1p(1 / n) / math.log(V) * (1 - 1e-12)))).sum())


# ------------------------------------------------------------ values in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
        H, o = case["H"], case["offset"]
        inv = lambda v: (torch.einsum("th,th->t", v, v) / H + EPS).pow(-0.5)  # noqa: E731
        if op == "norm_fwd":
            r = d["r"]
            out = []
            if case["block"]:
                n = torch.einsum("th,t,h->th", d["y"], inv(d["y"]), d["w_post"] + o) if case["post"] else d["y"]
                r = r + case["scale"] * (n if s["g"] is None else n * d["g"])
                out.append(r)
            return out + ([torch.einsum("th,t,h->th", r, inv(r), d["w_pre"] + o)] if case["pre"] else [])
        out, e = {}, d["dr_out"]
        if case["pre"]:  # d/dr of sum(dh * r * inv(r) * w): the product rule, inv' = -inv^3 r / H
            i, w = inv(d["r"]), d["w_pre"] + o
            a = torch.einsum("th,h,th->t", d["dh"], w, d["r"])
            e = e + d["dh"] * w * i[:, None] - d["r"] * (a * i ** 3 / H)[:, None]
            out["dw_pre"] = torch.einsum("th,th,t->h", d["dh"], d["r"], i)
        out["dr"] = e
        y, gate = d["y"], (d["g"] if s["g"] is not None else torch.ones((), dtype=torch.float64, device="cuda"))
        i, w = (inv(y), d["w_post"] + o) if case["post"] else (torch.ones_like(y[:, 0]), torch.ones_like(y[0]))
        u = case["scale"] * e * gate  # what reaches the normed rows
        if s["g"] is not None:
            dg = case["scale"] * e * y * i[:, None] * w
            out["dgate"] = {"token": lambda: dg.sum(1, keepdim=True), "channel": lambda: dg.sum(0), "element": lambda: dg}[case["gate"]]()
        out["dy"] = u * w * i[:, None]
        if case["post"]:
            out["dy"] = out["dy"] - y * (torch.einsum("th,h,th->t", u, w, y) * i ** 3 / H)[:, None]
            out["dw_post"] = torch.einsum("th,th,t->h", u, y, i)
        return out
    if op == "embed_fwd":
        return torch.index_select(s["table"], 0, s["ids"]).double() * s["scale"]
    if op == "embed_bwd":
        at, d = s["ids"].sort(stable=True)[1], s["dout"].double()
        if s["padding_id"] is not None:
            at = at[s["ids"][at] != s["padding_id"]]
        tokens, n = torch.unique_consecutive(s["ids"][at], return_counts=True)
        out = torch.zeros(case["V"], case["H"], dtype=torch.float64, device="cuda")
        for h in range(0, case["H"], 256):  # differences of running sums at the ends of the runs
            c = torch.cat([d.new_zeros(1, min(256, case["H"] - h)), d[:, h:h + 256][at].cumsum(0)])
            e = n.cumsum(0)
            out[tokens, h:h + 256] = (c[e] - c[e - n]) * s["scale"]
        return out
    T, tau = case["T"], case["tau"]
    losses, lses, grads = [], [], []
    for t in range(0, T, 2048):  # rows by rows, to keep the 64-bit copies small
        z = s["z"][t:t + 2048].double() / tau
        ids, tl = s["ids"][t:t + 2048].long(), s["t_logits"][t:t + 2048].double() / tau
        p = torch.softmax(tl.masked_fill(ids < 0, -math.inf), 1).nan_to_num(0.0)
        log_q = (z - (s["lse"][t:t + 2048].double() if op == "distill_bwd" else torch.logsumexp(z, 1))[:, None])
        at = torch.where(ids < 0, 0, ids)
        losses.append((torch.special.xlogy(p, p) - p * log_q.gather(1, at)).sum(1))
        lses.append(torch.logsumexp(z, 1))
        if op != "distill_fwd":
            k = s["weight"][t:t + 2048].double()[:, None] / tau
            grads.append((log_q.exp_() * (k * p.sum(1, keepdim=True))).scatter_add_(1, at, -k * p))
    if op == "distill_fwd":
        return torch.cat(losses), torch.cat(lses)
    if op == "distill_bwd":
        return torch.cat(grads)
    return torch.cat(losses), torch.cat(grads)
