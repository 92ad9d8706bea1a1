"""Plain 64-bit forms of the operators around the layer, for their tests.

Every reference returns its values with their magnitude: the same expression
with absolute values in the place of its terms, which is what a rounding error
is relative to.  A kernel output is then held to

    half an ulp of its type on the value  +  ops * 2^-24 on the magnitude

where ``ops`` counts the FP32 roundings a value goes through in the worst
case: ROW for outputs of a row (at most 32 elements a thread and 10 levels of
a tree for each statistic, of which a value has two, and some twenty single
operations), and one more for each term of a sum over rows.
"""
import torch

ROW = 128
U32 = 2.0 ** -24
HALF_ULP = {torch.float32: U32, torch.bfloat16: 2.0 ** -8}  # of 24 and 8 significant bits


def check(got, ref, mag, ops=ROW, what=""):
    """|got - ref| within the bound above; infinities and NaN in the same places."""
    g, r, m = got.double().cpu(), ref.double().cpu(), mag.double().cpu()
    assert g.shape == r.shape, f"{what}: {list(g.shape)} for {list(r.shape)}"
    fine = torch.isfinite(r)
    assert torch.equal(torch.isnan(g), torch.isnan(r)), f"{what}: NaN in other places"
    odd = ~fine & ~torch.isnan(r)
    assert torch.equal(g[odd], r[odd]), f"{what}: infinities in other places"
    m = torch.where(torch.isfinite(m), m, torch.full_like(m, float("inf")))
    tol = HALF_ULP[got.dtype] * r.abs() + (1 + HALF_ULP[got.dtype]) * ops * U32 * m + 1e-37
    bad = fine & ((g - r).abs() > tol)
    if bad.any():
        i = int(((g - r).abs() / tol).masked_fill(~fine, 0).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {r.numel()} off, worst at {i}: {g.flatten()[i]} for "
                             f"{r.flatten()[i]} (bound {tol.flatten()[i]})")


def norm(v, w, eps):
    rstd = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    return v * rstd * w, rstd


def block_norm(r, y, w_post, w_pre, gate, scale, eps, offset):
    """{name: (value, magnitude)} of r_out and h."""
    r = r.double()
    m, out = r.abs(), {}
    if y is not None:
        n = y.double()
        if w_post is not None:
            n = norm(n, w_post.double() + offset, eps)[0]
        n = scale * n * (1 if gate is None else gate.double())
        r, m = r + n, m + n.abs()
        out["r_out"] = (r, m)
    if w_pre is not None:
        w = w_pre.double() + offset
        h, rstd = norm(r, w, eps)
        out["h"] = (h, m * rstd * w.abs() + h.abs() * (r.abs() * m).mean(1, keepdim=True) * rstd ** 2)
    return out


def _norm_grad(d, v, w, rstd):
    x = v * rstd
    g = rstd * (d * w - x * (d * w * x).mean(1, keepdim=True))
    return g, rstd * ((d * w).abs() + x.abs() * (d * w * x).abs().mean(1, keepdim=True))


def block_norm_backward(dr_out, dh, r_out, y, w_post, w_pre, gate, scale, eps, offset):
    out = {}
    e = 0.0 if dr_out is None else dr_out.double()
    em = 0.0 if dr_out is None else e.abs()
    if w_pre is not None:
        v, w, d = r_out.double(), w_pre.double() + offset, dh.double()
        rstd = norm(v, w, eps)[1]
        g, gm = _norm_grad(d, v, w, rstd)
        e, em = e + g, em + gm
        x = d * v * rstd
        out["dw_pre"] = (x.sum(0), x.abs().sum(0))
    out["dr"] = (e, em)
    if y is None:
        return out
    v, gt = y.double(), (torch.ones((), dtype=torch.float64, device=y.device) if gate is None else gate.double())
    w = torch.ones(v.shape[1], dtype=torch.float64, device=y.device) if w_post is None else w_post.double() + offset
    rstd = torch.ones_like(v[:, :1]) if w_post is None else norm(v, w, eps)[1]
    u, um = scale * gt * e, abs(scale) * gt.abs() * em
    if gate is not None:
        dg, dgm = scale * e * v * rstd * w, abs(scale) * em * (v * rstd * w).abs()
        if gate.dim() == 1:
            dg, dgm = dg.sum(0), dgm.sum(0)
        elif gate.shape[1] == 1 and v.shape[1] != 1:
            dg, dgm = dg.sum(1, keepdim=True), dgm.sum(1, keepdim=True)
        out["dgate"] = (dg, dgm)
    if w_post is None:
        out["dy"] = (u, um)
        return out
    g = _norm_grad(u, v, w, rstd)[0]
    gm = rstd * ((um * w).abs() + (v * rstd).abs() * (um * w * v * rstd).abs().mean(1, keepdim=True))
    out["dy"] = (g, gm)
    x, xm = u * v * rstd, um * (v * rstd).abs()
    out["dw_post"] = (x.sum(0), xm.sum(0))
    return out


def embed(table, ids, scale):
    ok = (ids >= 0) & (ids < table.shape[0])
    out = table.double()[torch.where(ok, ids, 0).long()] * scale * ok[:, None]
    return out, out.abs()


def embed_backward(ids, dout, V, scale, padding_id=None):
    keep = (ids >= 0) & (ids < V)
    if padding_id is not None:
        keep &= ids != padding_id
    d = dout.double()[keep] * scale
    out = torch.zeros(V, dout.shape[1], dtype=torch.float64, device=dout.device)
    return out.index_add(0, ids[keep].long(), d), out.index_add(0, ids[keep].long(), d.abs())


def distill(logits, t_ids, t_logits, tau=1.0, scale=1.0, t_lse=None, weight=None):
    """{name: (value, magnitude)} of loss, lse and (with weight) dlogits."""
    z, t = logits.double() / tau, t_logits.double() / tau
    there = (t_ids >= 0) & (t_ids < z.shape[1]) & (t != -float("inf"))
    t = t.masked_fill(~there, -float("inf"))
    c = torch.logsumexp(t, 1) if t_lse is None else t_lse.double()
    p = torch.where(there, torch.exp(t - c[:, None]), 0.0)
    logp = torch.where(p > 0, t - c[:, None], 0.0)
    lse = torch.logsumexp(z, 1)
    at = torch.where(there, t_ids, 0).long()
    zk = z.gather(1, at)
    term = torch.where(p > 0, p * (logp - (zk - lse[:, None])), 0.0)
    any_, none = there.any(1), lse == -float("inf")
    loss = torch.where(any_, torch.where(none, float("inf"), term.sum(1)), 0.0) * scale
    # roundings of an exponent are absolute: relative to the largest term of it
    size = 1 + z.abs().masked_fill(z.isinf(), 0).amax(1) + t.abs().masked_fill(t.isinf(), 0).amax(1) + \
        torch.where(lse.isinf(), 0.0, lse.abs()) + (0 if t_lse is None else t_lse.double().abs())
    out = {"loss": (loss, any_ * abs(scale) * p.sum(1) * size * (1 + size)), "lse": (lse, size)}
    if weight is not None:
        w = weight.double()
        live = any_ & ~none & (w != 0)
        k = (w * scale / tau)[:, None]
        q = torch.exp(z - lse[:, None])
        total = p.sum(1, keepdim=True)
        d = (q * total).scatter_add(1, at, -p) * k
        m = (q * total).scatter_add(1, at, p) * k.abs() * (1 + size[:, None])
        z0 = torch.zeros_like(d)
        out["dlogits"] = (torch.where(live[:, None], d, z0), torch.where(live[:, None], m, z0))
    return out
