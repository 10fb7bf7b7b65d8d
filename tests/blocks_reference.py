"""Plain 64-bit forms of the embedding, layer norm and gated operators, and the
error each may have: derived from the roundings the operators state, before any
comparison."""
import torch

import residual_reference as R
from residual_reference import EPS32, rounded


def lookup(table, ids, scale, dtype):
    """(rows, error after the one rounding)."""
    t, i = table.double().cpu(), ids.cpu().long()
    known = (i >= 0) & (i < t.shape[0])
    y = torch.zeros(i.shape[0], t.shape[1], dtype=torch.float64)
    y[known] = t[i[known]] * scale
    return y, rounded(y, EPS32 * y.abs(), dtype)


def lookup_grad(dy, ids, rows, scale):
    """(gradient, error before its rounding): fp32 sums of as many rows as share an id, and the product with scale."""
    d, i = dy.double().cpu(), ids.cpu().long()
    known = (i >= 0) & (i < rows)
    d, i = d[known], i[known]
    total = torch.zeros(rows, dy.shape[1], dtype=torch.float64).index_add_(0, i, d)
    size = torch.zeros_like(total).index_add_(0, i, d.abs())
    count = torch.bincount(i, minlength=rows).double()[:, None]
    return total * scale, abs(scale) * ((count + 2) * EPS32 * size + EPS32 * total.abs())


def layer_norm(x, r, w, b, eps):
    """(s, mean, q, y, their errors in fp32 as a tuple of the last three's)."""
    s = x.double().cpu() + (0 if r is None else r.double().cpu())
    c = s.shape[1]
    one = torch.ones(c, dtype=torch.float64)
    w = one if w is None else w.double().cpu()
    b = 0 * one if b is None else b.double().cpu()
    mu = s.mean(1, keepdim=True)
    e_mu = (c + 4) * EPS32 * s.abs().mean(1, keepdim=True)
    d = s - mu
    e_d = e_mu + EPS32 * (s.abs() + mu.abs())
    var = d.square().mean(1, keepdim=True)
    # a shifted mean moves the mean square of the differences by its own square only: sum d = 0
    e_var = e_mu.square() + 2 * (d.abs() * EPS32 * (s.abs() + mu.abs())).mean(1, keepdim=True) + (c + 4) * EPS32 * (var + e_mu.square())
    q = (var + eps).rsqrt()
    e_q = q * (0.5 * e_var / (var + eps) * (1 + e_var / (var + eps)) + 4 * EPS32)
    y = d * q * w + b
    e_y = w.abs() * (q * e_d + (d.abs() + e_d) * e_q) + 4 * EPS32 * ((d * q * w).abs() + b.abs())
    return s, mu[:, 0], q[:, 0], y, (e_mu[:, 0], e_q[:, 0], e_y)


def layer_norm_grad(dy, s, w, mu, q, ds):
    """[(value, error before its rounding)] of dx, dw, db."""
    dy, s = dy.double().cpu(), s.double().cpu()
    mu, q = mu.double().cpu()[:, None], q.double().cpu()[:, None]
    m, c = s.shape
    w = torch.ones(c, dtype=torch.float64) if w is None else w.double().cpu()
    h, g = (s - mu) * q, dy * w
    e_h = 2 * EPS32 * (s.abs() + mu.abs()) * q.abs()
    mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    e_mg = (c + 4) * EPS32 * g.abs().mean(1, keepdim=True)
    e_mgh = (g.abs() * e_h).mean(1, keepdim=True) + (c + 8) * EPS32 * (g * h).abs().mean(1, keepdim=True)
    dx = q * (g - mg - h * mgh)
    ex = q * (e_mg + h.abs() * e_mgh + e_h * mgh.abs() + 4 * EPS32 * (g.abs() + mg.abs() + (h * mgh).abs()))
    if ds is not None:
        dx = dx + ds.double().cpu()
        ex = ex + EPS32 * dx.abs()
    dw = (dy * h).sum(0), (dy.abs() * e_h).sum(0) + (m + 8) * EPS32 * (dy * h).abs().sum(0)
    return (dx, ex), dw, (dy.sum(0), (m + 8) * EPS32 * dy.abs().sum(0))


def argument(z, kind):
    """Size of the logistic's argument (see residual_reference.linear)."""
    return (z.abs() if kind == "silu" else 1.6 * z.abs() * (1 + 0.045 * z * z)).clamp_max(100)


def act_error(z, ez, kind):
    """Error of act(z), z known to within ez (as in residual_reference.linear)."""
    if kind in ("none", "relu"):
        return ez
    return 1.2 * ez + R.act(z, kind).abs() * (4 * argument(z, kind) + 8) * EPS32


def gated(x, wg, wu, bg, bu, kind, xs, gs, us, dtype):
    """(h, g, u, error of h, errors of g and u before their rounding)."""
    _, g, _, eg = R.linear(x, wg, bg, "none", None, xs, gs, torch.float32)
    _, u, _, eu = R.linear(x, wu, bu, "none", None, xs, us, torch.float32)
    a, ea = R.act(g, kind), act_error(g, eg, kind)
    h = a * u
    return h, g, u, rounded(h, (a.abs() + ea) * eu + u.abs() * ea + EPS32 * h.abs(), dtype), eg, eu


def gated_grad(dh, x, wg, wu, g, u, kind):
    """[(value, error before its rounding)] of dx, dwg, dwu, dbg, dbu."""
    dtype = x.dtype
    dh, x, wg, wu, g, u = (t.double().cpu() for t in (dh, x, wg, wu, g, u))
    a, s = R.act(g, kind), R.slope(g, kind)
    dg, du = dh * u * s, dh * a
    steps = 0 if kind in ("none", "relu") else 4 * argument(g, kind)
    # the slope p + t p (1 - p) and the value z p: each factor to a few ulps of its size, p's argument as in argument()
    eg = (dh * u).abs() * (steps + 16) * EPS32 * (1.2 if kind not in ("none", "relu") else s) + 2 * EPS32 * dg.abs()
    eu = du.abs() * (steps + 8) * EPS32
    rg, ru = rounded(dg, eg, dtype), rounded(du, eu, dtype)
    m, n = dg.shape
    bg, bu = dg.abs() + rg, du.abs() + ru
    dx = dg @ wg + du @ wu
    ex = rg @ wg.abs() + ru @ wu.abs() + (2 * n + 4) * EPS32 * (bg @ wg.abs() + bu @ wu.abs())
    out = [(dx, ex)]
    for d, r, big in ((dg, rg, bg), (du, ru, bu)):
        out.append((d.t() @ x, r.t() @ x.abs() + (m + 4) * EPS32 * (big.t() @ x.abs())))
    for d, e in ((dg, eg), (du, eu)):
        out.append((d.sum(0), e.sum(0) + (m + 4) * EPS32 * (d.abs() + e).sum(0)))
    return out


def check_8bit(y, scale, want, err):
    """An 8-bit row: a code is within half its step (2^-4 of the value, 2^-10 of the scale below 2^-6) of its value."""
    at = want.abs().argmax(1, keepdim=True)
    top, e_top = want.abs().gather(1, at)[:, 0], err.amax(1)
    sc = scale.double().cpu()
    assert ((sc - top / 448).abs() <= e_top / 448 + 4 * EPS32 * top / 448).all()
    rel = (e_top / top.clamp_min(1e-300))[:, None] + 8 * EPS32
    R.within(y.float().double().cpu() * sc[:, None], want, want.abs() * (2.0 ** -4 + 2 * rel) + 1.1 * err + 2.0 ** -10 * sc[:, None] * (1 + 4 * rel))
