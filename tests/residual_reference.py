"""Plain 64-bit forms of the residual head's operators, and the error each may
have: derived from the roundings the operators state, before any comparison."""
import math

import torch

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a unit in the last place
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149}  # half the smallest subnormal
EPS32 = 2.0 ** -23  # a step of an fp32 sum on the matrix cores, rounded either way


def act(z, kind):
    if kind == "relu":
        return z.clamp_min(0)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope(z, kind):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0).double()
    if kind == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)


def rounded(y, err, dtype):
    """Error of a value known to within err, rounded once to dtype."""
    return err + UNIT[dtype] * (y.abs() + err) + TINY[dtype]


def linear(x, w, b, kind, r, xs, ws, dtype):
    """(y, z, error of y, error of z before its rounding)."""
    x, w = x.double().cpu(), w.double().cpu()
    if xs is not None:
        x, w = x * xs.double().cpu()[:, None], w * ws.double().cpu()[:, None]
    z, size = x @ w.t(), x.abs() @ w.abs().t()
    if b is not None:
        z, size = z + b.double().cpu(), size + b.double().cpu().abs()
    ez = (x.shape[1] + 4) * EPS32 * size
    a = act(z, kind)
    ea = ez
    if kind in ("silu", "gelu_tanh"):
        # slopes stay below 1.13; the logistic's argument u (|u| <= |z| or 1.6 |z| (1 + z^2 / 20)) is rounded a few
        # times, which moves it by a few ulps of u, and its exponential, sum and reciprocal round to an ulp each
        u = z.abs() if kind == "silu" else 1.6 * z.abs() * (1 + 0.045 * z * z)
        ea = 1.2 * ez + a.abs() * (4 * u.clamp_max(100) + 8) * EPS32
    y = a
    if r is not None:
        y = y + r.double().cpu()
        ea = ea + EPS32 * (y.abs() + a.abs())
    return y, z, rounded(y, ea, dtype), ez


def dz(dy, pre, kind, dtype):
    """(dz, error of its fp32 value, error after its rounding to the operands' type)."""
    d = dy.double().cpu()
    if kind == "none":
        e = torch.zeros_like(d)
        return d, e, (UNIT[dtype] * d.abs() + TINY[dtype] if dy.dtype == torch.float32 else e)
    z = pre.double().cpu()
    s = slope(z, kind)
    v = d * s
    # s = p + z p (1 - p) c: each term to a few ulps of its size, the argument of p as in linear()
    u = z.abs() if kind == "silu" else 1.6 * z.abs() * (1 + 0.045 * z * z)
    e = torch.zeros_like(v) if kind == "relu" else d.abs() * (4 * u.clamp_max(100) + 16) * EPS32 * 1.2
    return v, e, rounded(v, e, dtype)


def linear_grad(dy, x, w, pre, kind):
    """[(value, error before its rounding)] of dx, dw, db."""
    dtype = x.dtype
    v, e, er = dz(dy, pre, kind, dtype)
    m, n = v.shape
    x, w = x.double().cpu(), w.double().cpu()
    big = v.abs() + er
    dx = v @ w, er @ w.abs() + (n + 4) * EPS32 * (big @ w.abs())
    dw = v.t() @ x, er.t() @ x.abs() + (m + 4) * EPS32 * (big.t() @ x.abs())
    return dx, dw, (v.sum(0), e.sum(0) + (m + 4) * EPS32 * (v.abs() + e).sum(0))


def norm(x, r, w, eps):
    """(s, 1 / rms, y, relative error of y in fp32)."""
    s = x.double().cpu() + (0 if r is None else r.double().cpu())
    q = (s.square().mean(1) + eps).rsqrt()
    # sum of c squares (half of its relative error reaches q), s itself, q's root and reciprocal, two products
    return s, q, s * q[:, None] * w.double().cpu(), (s.shape[1] / 2 + 10) * EPS32


def norm_grad(dy, s, w, q, ds):
    """[(value, error before its rounding)] of dx, dw."""
    dy, s, w, q = (t.double().cpu() for t in (dy, s, w, q))
    c, m = s.shape[1], s.shape[0]
    h = s * q[:, None]
    g = dy * w
    dot = (g * h).mean(1, keepdim=True)
    size = (g * h).abs().mean(1, keepdim=True)
    dx = q[:, None] * (g - h * dot)
    ex = q[:, None] * (4 * EPS32 * g.abs() + h.abs() * (c + 8) * EPS32 * size)
    if ds is not None:
        dx = dx + ds.double().cpu()
        ex = ex + EPS32 * dx.abs()
    return (dx, ex), ((dy * h).sum(0), (m + 8) * EPS32 * (dy * h).abs().sum(0))


def within(got, want, err):
    d = (got.double().cpu() - want).abs()
    bad = ~(d <= err)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((d - err).max()):.3g} past its bound " \
                          f"at {bad.nonzero()[0].tolist()}: {got.cpu()[tuple(bad.nonzero()[0])].item()} for {want[tuple(bad.nonzero()[0])].item()}"
