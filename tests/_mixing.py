"""Group norm and window attention in 64 bits (torch, CPU), written from their
formulas, with bounds on how far float32 arithmetic, roundings of matrix operands
to 16 bits and one rounding of the output may be from them (u = 2^-24, gamma(n) as
in _rowops).

Group norm. Additions run in chains of at most `chain` terms: a thread's rows of a
piece, the threads of a block, the channels of a group, the pieces of a sample. The
sums are of differences from a row of the sample, so of at most `far` (the largest
distance of two values of a group), which bounds the mean's error by gamma(chain)
far and the variance's by gamma(chain + 8) far^2.

Attention. Scores are float32 sums of exact products; P (and dS) are rounded to the
rows' type on their way into the second product, half an ulp each."""
import math

import torch

import _rowops as ro

U = ro.U


def chain(n, c, groups):
    """Longest chain of additions: 1024 threads a block, 256 blocks."""
    words = -(-c // 8)
    a_thread = 2 * max(n * words / 2.0 ** 18, 4) + 2
    return int(a_thread + 10 + (c // groups) / 64 + 7 + 258 * (groups + 1023) / 1024 + 11) + 8


def runs(offsets, n):
    return [(0, n)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def group_stats(x, groups, offsets, eps):
    """float64 (mean, rstd, bound of mean, relative bound of rstd), each [samples, groups]."""
    n, c = x.shape
    out = []
    g = ro.gamma(chain(n, c, groups) + 8)
    for begin, end in runs(offsets, n):
        if begin == end:
            out.append(torch.zeros(4, groups, dtype=torch.float64))
            continue
        v = x[begin:end].reshape(end - begin, groups, -1).transpose(0, 1).reshape(groups, -1)
        mean, var = v.mean(1), v.var(1, unbiased=False)
        far = v.amax(1) - v.amin(1)
        rstd = torch.where(var + eps > 0, (var + eps) ** -0.5, torch.zeros_like(var))
        # d rstd / rstd = - d var / (2 (var + eps)); sums, root and division add 4 u
        rel = g * far ** 2 / (2 * (var + eps)).clamp(min=1e-300) + 4 * U
        out.append(torch.stack((mean, rstd, g * far + 2 * U * mean.abs(), rel)))
    return torch.stack(out, 1).unbind(0)


def spread(t, x, offsets, groups):
    """[samples, groups] -> a value for each element of x, zeros in rows of no sample."""
    n, c = x.shape
    rows = torch.zeros(n, groups, dtype=torch.float64)
    for k, (begin, end) in enumerate(runs(offsets, n)):
        rows[begin:end] = t[k]
    return rows.repeat_interleave(c // groups, 1)


def inside(x, offsets):
    n = x.shape[0]
    at = torch.arange(n)[:, None]
    return ((at >= offsets[0]) & (at < offsets[-1])).double() if offsets is not None else torch.ones(n, 1, dtype=torch.float64)


def group_norm(x, w, b, groups, offsets, eps, name, dt):
    """float64 (y, bound)."""
    mean, rstd, em, er = group_stats(x, groups, offsets, eps)
    mean, rstd, em, er = (spread(t, x, offsets, groups) for t in (mean, rstd, em, er))
    xh = (x - mean) * rstd
    z = xh * w + b
    ez = w.abs() * (rstd * em + xh.abs() * (er + 3 * U) + 2 * U * rstd * mean.abs()) + 3 * U * (z.abs() + b.abs())
    v = ro.act(z, name)
    err = 1.13 * ez + ro.eval_err(z, v) * (name not in (None, "none", "relu"))
    keep = inside(x, offsets)
    return v * keep, ro.rounded(v, err, dt)


def group_norm_backward(dy, x, w, b, groups, stats, offsets, name, dt):
    """((dx, bound), (dw, bound), (db, bound)) for float32 statistics taken as they are."""
    n, c = x.shape
    keep = inside(x, offsets)
    mean, rstd = (spread(stats[:, :, k], x, offsets, groups) for k in (0, 1))
    xh = (x - mean) * rstd
    exh = 3 * U * (x.abs() + mean.abs()) * rstd
    z = xh * w + b
    ez = w.abs() * exh + 3 * U * (z.abs() + b.abs())
    dz = dy * ro.slope(z, name) * keep
    soft = name not in (None, "none", "relu")
    edz = dy.abs() * soft * (1.1 * ez + 2.0 ** -20 * (1 + z.abs())) + 2 * U * dz.abs()
    a, ea = dz * w, edz * w.abs() + U * (dz * w).abs()
    g = ro.gamma(chain(n, c, groups))

    def means(v, e):
        """Mean over each sample and group, and its bound, an element each."""
        total, bound = [], []
        for begin, end in runs(offsets, n):
            size = max(1, (end - begin) * (c // groups))
            total.append(v[begin:end].reshape(end - begin, groups, c // groups).sum((0, 2)) / size)
            bound.append((e + g * v.abs())[begin:end].reshape(end - begin, groups, c // groups).sum((0, 2)) / size)
        return [spread(torch.stack(t), x, offsets, groups) for t in (total, bound)]

    m1, em1 = means(a, ea)
    m2, em2 = means(a * xh, ea * xh.abs() + a.abs() * exh + U * (a * xh).abs())
    dx = rstd * (a - m1 - xh * m2)
    ex = rstd * (ea + em1 + xh.abs() * em2 + exh * m2.abs() + 6 * U * (a.abs() + m1.abs() + (xh * m2).abs()))
    dw, ew = (dz * xh).sum(0), (edz * xh.abs() + dz.abs() * exh + g * (dz * xh).abs()).sum(0)
    db, eb = dz.sum(0), (edz + g * dz.abs()).sum(0)
    return [(v, ro.rounded(v, e, dt)) for v, e in ((dx, ex), (dw, ew), (db, eb))]
