"""The row operators in 64 bits (torch, CPU), written from their formulas, with
bounds on how far float32 arithmetic and one rounding may be from them.

Bounds. u = 2^-24. A float32 sum of n products in any order is within
gamma(n) sum |terms| of the exact one. An activation is 1.13-Lipschitz at most
(gelu's slope; silu 1.10) and is computed to 2^-20 of |z| + |value| (exp, erf
and reciprocal to a few ulp). An output of type T adds half an ulp: 2^-8 |y|
(bf16) or 2^-11 |y| + 2^-25 (f16). Slopes: |act'| <= 1.13, and 1.1-Lipschitz
(silu and gelu; the second derivatives are below 0.8); relu's slope jumps at 0,
so rows near it are left out by the caller or given exact inputs.

e4m3 products. The instruction adds groups of 8 consecutive products aligned to
the largest of the group, with 13 bits below its leading bit kept (measured:
beside +-2^16 a product of 2^3 counts and one of 2^2 does not, in the same
group of 8; between groups and in the accumulator 24 bits are kept). Each of
the 7 others loses less than 2^-13 of the largest: E4M3_LOSS of sum |terms|.
"""
import math

import torch

U = 2.0 ** -24
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}     # 8 and 11 significant bits
FLOOR = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
E4M3 = torch.float8_e4m3fn
E4M3_LOSS = 7 * 2.0 ** -13


def gamma(n):
    return n * U / (1 - n * U)


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2.0)))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2.0))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def pre(x, w, bias, extra_terms=2, loss=0.0):
    """(z, bound on |float32 z - z|) of z = x w + bias, float64 operands."""
    z = x @ w
    mag = x.abs() @ w.abs()
    lost = loss * mag
    if bias is not None:
        z, mag = z + bias, mag + bias.abs()
    return z, gamma(x.shape[1] + extra_terms) * mag + lost


def eval_err(z, v):
    return 2.0 ** -20 * (z.abs() + v.abs())


def rounded(y, err, dt):
    """Bound on |T(float32 y) - y| where the float32 y is within err."""
    return err + HALF_ULP[dt] * (y.abs() + err) * 1.01 + FLOOR[dt]


def check(got, want, bound, label):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, f"{label}: shape {tuple(got.shape)} != {tuple(want.shape)}"
    if got.numel() == 0:
        return
    over = (got - want).abs() - bound
    bad = ~(over <= 0)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {got.numel()} outside the bound, first at "
                             f"{i}: got {got[i].item()}, want {want[i].item()}, bound {bound[i].item()}")


def linear(x, w, bias, residual, name, dt):
    """float64 (y, bound)."""
    z, ez = pre(x, w, bias)
    v = act(z, name)
    err = 1.13 * ez + eval_err(z, v) * (name not in (None, "none", "relu"))
    y = v
    if residual is not None:
        y = v + residual
        err = err + U * y.abs()
    return y, rounded(y, err, dt)


def gated(x, w, bias, name, dt):
    z, ez = pre(x, w, bias)
    f = z.shape[1] // 2
    g, u, eg, eu = z[:, :f], z[:, f:], ez[:, :f], ez[:, f:]
    a = act(g, name)
    ea = 1.13 * eg + eval_err(g, a)
    y = a * u
    err = ea * u.abs() + a.abs() * eu + ea * eu + 2 * U * y.abs()
    return y, rounded(y, err, dt)


def gradients(dz, edz, x, w, dt):
    """dx, dw, db and their bounds for a 16-bit dz within edz (its rounding
    included) of the exact one."""
    n, c = x.shape
    wide = dz.shape[1]
    mag = dz.abs() + edz
    dx = dz @ w.t()
    ex = edz @ w.abs().t() + gamma(wide + 2) * (mag @ w.abs().t())
    dw = x.t() @ dz
    ew = x.abs().t() @ edz + gamma(n + 2) * (x.abs().t() @ mag)
    db = dz.sum(0)
    eb = edz.sum(0) + gamma(n + 2) * mag.sum(0)
    return [(v, rounded(v, e, dt)) for v, e in ((dx, ex), (dw, ew), (db, eb))]


def linear_backward(dy, x, w, bias, name, dt):
    z, ez = pre(x, w, bias)
    if name in (None, "none"):
        return gradients(dy, torch.zeros_like(dy), x, w, dt)
    s = slope(z, name)
    dz = dy * s
    e = dy.abs() * (1.1 * ez + 2.0 ** -20 * (1 + z.abs())) * (name != "relu")
    return gradients(dz, rounded(dz, e, dt), x, w, dt)


def gated_backward(dh, x, w, bias, name, dt):
    z, ez = pre(x, w, bias)
    f = z.shape[1] // 2
    g, u, eg, eu = z[:, :f], z[:, f:], ez[:, :f], ez[:, f:]
    a, s = act(g, name), slope(g, name)
    soft = name != "relu"
    es = (1.1 * eg + 2.0 ** -20 * (1 + g.abs())) * soft
    ea = 1.13 * eg + eval_err(g, a)
    dz = torch.cat((dh * u * s, dh * a), 1)
    e = torch.cat((dh.abs() * (u.abs() * es + eu * (s.abs() + es)) + 3 * U * (dh * u * s).abs(),
                   dh.abs() * ea + 2 * U * (dh * a).abs()), 1)
    return gradients(dz, rounded(dz, e, dt), x, w, dt)


def norm(x, residual, w, eps):
    """float64 (y, relative-error bound of the float32 y, s)."""
    s = x if residual is None else x + residual
    c = s.shape[1]
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * w
    # s is rounded (1 u), the mean's relative error is gamma(c + 3), halved by the
    # root; root, division and two products: 5 more roundings
    rel = U + 0.5 * gamma(c + 5) + 6 * U
    return y, rel, s


def norm_backward(dy, s, w, eps, ds, dt):
    n, c = s.shape
    rstd = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    xh = s * rstd
    a = dy * w
    m = (a * xh).mean(1, keepdim=True)
    dx = rstd * (a - xh * m)
    rel = 0.5 * gamma(c + 5) + 4 * U                 # of rstd and x_hat
    mag = rstd * (a.abs() + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    ex = (gamma(c + 8) + 3 * rel) * mag
    if ds is not None:
        dx = dx + ds
        ex = ex + U * dx.abs()
    dw = (dy * xh).sum(0)
    ew = (gamma(n + 4) + rel) * (dy * xh).abs().sum(0)
    return (dx, rounded(dx, ex, dt)), (dw, rounded(dw, ew, dt))
