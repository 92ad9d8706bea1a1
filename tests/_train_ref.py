"""Plain 64-bit forms of the end of a training step, with the bounds that the
kernels are held to.

With u = half an ulp of the outputs' type (2^-8 for bfloat16, 2^-24 for
float32) and v = 2^-24:

a logit       sums D exact products in FP32: an error of at most (D + 8) * 2 v
              times the sum of their magnitudes (2 v an addition, since the
              tensor cores cut off where others round), dx in all.  Eight more for the
              scaling and the passage to base 2.
lse, loss     the largest dx of a row twice (once in lse, once in the target),
              the sum of exponentials (2^-22 each from the instruction, V / 64 + 16
              additions of positive terms in a chain at most 64 + V / 64 long), and
              a few roundings of lse itself.
g             relative to its two terms: p = exp(x - lse) is off by dp = dx + 8 v |lse| +
              2^-21; in bfloat16 every entry is rounded once (u) but the target's.
dhidden       the rounding of g over the sum of magnitudes |g| |w|, dp over that of p |w|, FP32 sums
              (gamma: V roundings, chopped: 2 v each), u on the result.
dweight       the same over the rows, with one rounding more (u) in bfloat16 for the
              row of hidden over its factor.
"""
import torch

V24 = 2.0 ** -24
U = {torch.float32: V24, torch.bfloat16: 2.0 ** -8}
IGNORE = -100


def cross_entropy(h, w, t, dloss, scale=1.0, z=0.0, lse=None):
    """Values and bounds: {name: (value, bound)} of loss, lse, dhidden, dweight."""
    u16 = U[torch.bfloat16] if h.dtype is torch.bfloat16 else 0.0
    out_u = U[h.dtype]
    V, D = w.shape
    keep = (t >= 0) & (t < V) & (t != IGNORE)
    h, w = torch.where(keep[:, None], h.double(), 0.0), w.double()
    t = torch.where(keep, t.long(), 0)
    x = scale * (h @ w.t())
    dx = abs(scale) * (h.abs() @ w.abs().t()) * ((D + 8) * 2 * V24)
    own = lse is None
    lse = torch.logsumexp(x, 1) if own else lse.double()
    row = dx.amax(1)
    xt = x.gather(1, t[:, None])[:, 0]
    l_tol = row + (64 + V / 64 + 16) * V24 + 2.0 ** -22 + 8 * V24 * lse.abs()
    loss = lse - xt + z * lse * lse
    loss_tol = 2 * row + l_tol * (1 + 2 * z * lse.abs()) + 4 * V24 * loss.abs() + 4 * V24 * z * lse * lse
    out = {"loss": (torch.where(keep, loss, 0.0), torch.where(keep, loss_tol, 0.0)),
           "lse": (torch.where(keep, lse, 0.0), torch.where(keep, l_tol, 0.0))}
    d = torch.where(keep, dloss.double(), 0.0) * scale
    p = torch.exp(x - lse[:, None]) * (d * (1 + 2 * z * lse))[:, None]
    g = p.clone()
    g.scatter_add_(1, t[:, None], -d[:, None])
    dp = (dx + row[:, None] + 8 * V24 * lse.abs()[:, None] + 2.0 ** -21 + (l_tol[:, None] if own else 0.0)) * 1.1
    e = p.abs() * dp + g.abs() * 8 * V24  # error of g before its rounding
    off = (g.abs() + e) * (u16 * 1.01)
    off.scatter_(1, t[:, None], 0.0)      # (the target's entry is exact)
    off = off + e
    dh, dw = g @ w, g.t() @ h
    n_h, n_w = (V + 8) * 2 * V24, (h.shape[0] + 8) * 2 * V24
    dh_tol = off @ w.abs() + n_h * (g.abs() @ w.abs())
    dw_tol = off.t() @ h.abs() + (n_w + 1.02 * u16) * (g.abs().t() @ h.abs())
    out["dhidden"] = (dh, dh_tol * 1.01 + out_u * 1.01 * dh.abs() + 1e-37)
    out["dweight"] = (dw, dw_tol * 1.01 + out_u * 1.01 * dw.abs() + 1e-37)
    out["dweight32"] = (dw, dw_tol * 1.01 + V24 * dw.abs() + 1e-37)
    return out


def check(got, ref, what):
    value, tol = ref
    assert got.shape == value.shape, (what, got.shape, value.shape)
    bad = ~((got.double() - value).abs() <= tol)
    if bad.any():
        off = ((got.double() - value).abs() / tol.clamp_min(1e-300))
        i = int(torch.where(torch.isnan(off), float("inf"), off).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, worst at {i}: {float(got.flatten()[i])} for "
                             f"{float(value.flatten()[i])} (bound {float(tol.flatten()[i])})")
