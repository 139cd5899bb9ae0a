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
    """Longest chain of additions: 512 threads a block, 512 blocks and one more a sample."""
    words = -(-c // 8)
    a_thread = 2 * max(n * words / 2.0 ** 18, 4) + 2
    return int(a_thread + 10 + (c // groups) / 64 + 7 + 516 * (groups + 511) / 512 + 11) + 8


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


# ---- window attention --------------------------------------------------------------


def scores(q, k, coords, table, heads, kv, scale):
    """float64 scores [heads, L, L] of one window, the bound of float32's, and the heads' keys."""
    length, dim = q.shape[0], q.shape[1] // heads
    q = q.view(length, heads, dim).transpose(0, 1)
    k = k.view(length, kv, dim).transpose(0, 1).repeat_interleave(heads // kv, 0)
    s = scale * (q @ k.transpose(1, 2))
    err = ro.gamma(dim + 4) * scale * (q.abs() @ k.abs().transpose(1, 2))
    if table is not None:
        r = table.shape[1] // 2
        apart = (coords[:, None] - coords[None]).clamp(-r, r) + r
        for axis in range(3):
            t = table[axis][apart[:, :, axis]].permute(2, 0, 1)
            s, err = s + t, err + 4 * U * t.abs()
    return s, err + 4 * U * s.abs(), q, k


def window_rows(offsets, order, n):
    """(places, rows) of each window."""
    order = torch.arange(n) if order is None else order.long()
    return [(slice(b, e), order[b:e]) for b, e in zip(offsets[:-1], offsets[1:]) if e > b]


def attention(q, k, v, offsets, order, coords, table, heads, kv, scale, dt):
    """float64 (out, bound, lse by place, bound)."""
    n, dim = q.shape[0], q.shape[1] // heads
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((heads, n), -math.inf, dtype=torch.float64)
    el = torch.zeros((heads, n), dtype=torch.float64)
    for places, rows in window_rows(offsets, order, n):
        length = len(rows)
        s, es, _, _ = scores(q[rows], k[rows], None if coords is None else coords[rows], table, heads, kv, scale)
        vw = v[rows].view(length, kv, dim).transpose(0, 1).repeat_interleave(heads // kv, 0)
        top = s.amax(2, keepdim=True)
        total = torch.exp(s - top).sum(2, keepdim=True)
        p = torch.exp(s - top) / total
        # an exponential: its argument's error, and 2^-21 of itself for the function and its base
        ep = 2 * es.amax(2, keepdim=True) + 4 * U * (s.abs().amax(2, keepdim=True) + top.abs()) + 2.0 ** -21
        mag = p @ vw.abs()
        e = mag * (2 * ep + ro.HALF_ULP[dt] + ro.gamma(2 * length + 80))
        if dt == torch.float16:             # P below f16's normal range
            e = e + ro.FLOOR[dt] * vw.abs().sum(1, keepdim=True)
        o = p @ vw
        out[rows] = o.transpose(0, 1).reshape(length, -1)
        bound[rows] = ro.rounded(o, e, dt).transpose(0, 1).reshape(length, -1)
        lse[:, places] = (top + torch.log(total)).squeeze(2)
        el[:, places] = (ep + ro.gamma(length + 80)).squeeze(2) + 4 * U * lse[:, places].abs()
    return out, bound, lse, el


def attention_backward(dout, q, k, v, offsets, order, coords, table, heads, kv, scale, dt):
    """[(gradient, bound)] of q, k, v and the table, for out and lse rounded to dt and float32."""
    n, dim = q.shape[0], q.shape[1] // heads
    hulp, each = ro.HALF_ULP[dt], heads // kv
    grads = [torch.zeros_like(t) for t in (q, k, v)]
    errs = [torch.zeros_like(t) for t in (q, k, v)]
    dtable = torch.zeros_like(table) if table is not None else None
    et, mt = (torch.zeros_like(table), torch.zeros_like(table)) if table is not None else (None, None)

    def joined(t, shared):
        t = t.view(kv, each, *t.shape[1:]).sum(1) if shared else t
        return t.transpose(0, 1).reshape(t.shape[1], -1)

    for _, rows in window_rows(offsets, order, n):
        length = len(rows)
        c = None if coords is None else coords[rows]
        s, es, qw, kw = scores(q[rows], k[rows], c, table, heads, kv, scale)
        vw = v[rows].view(length, kv, dim).transpose(0, 1).repeat_interleave(each, 0)
        do = dout[rows].view(length, heads, dim).transpose(0, 1)
        lse = torch.logsumexp(s, 2, keepdim=True)
        p = torch.exp(s - lse)
        ep = es + 4 * U * (s.abs() + lse.abs()) + 2.0 ** -21
        dp = do @ vw.transpose(1, 2)
        o = p @ vw
        delta = (do * o).sum(2, keepdim=True)
        edp = ro.gamma(dim + 4) * (do.abs() @ vw.abs().transpose(1, 2))
        edelta = (do.abs() * o.abs()).sum(2, keepdim=True) * (hulp + ro.gamma(dim + 4))
        ds = p * (dp - delta)
        eds = p * (edp + edelta) + (ep + hulp + 4 * U) * ds.abs()
        pe = p * (ep + hulp)
        if dt == torch.float16:
            # dS is taken times a power of two that brings 2 dim max |dout| max |v| to 2^14 or more
            eds = eds + dim * do.abs().max() * vw.abs().max() * 2.0 ** -38
            pe = pe + ro.FLOOR[dt]
        g = ro.gamma(length * each + 80)
        mag = ds.abs() + eds
        for i, (val, err, shared) in enumerate((
                (scale * (ds @ kw), scale * ((eds + g * mag) @ kw.abs()), False),
                (scale * (ds.transpose(1, 2) @ qw), scale * ((eds + g * mag).transpose(1, 2) @ qw.abs()), True),
                (p.transpose(1, 2) @ do, (pe + g * p).transpose(1, 2) @ do.abs(), True))):
            grads[i][rows], errs[i][rows] = joined(val, shared), joined(err, shared)
        if table is not None:
            r = table.shape[1] // 2
            apart = (c[:, None] - c[None]).clamp(-r, r) + r
            for axis in range(3):
                at = apart[:, :, axis].flatten()
                for to, t in ((dtable, ds), (et, eds), (mt, mag)):
                    to[axis].index_add_(0, at, t.permute(1, 2, 0).reshape(-1, heads))
    out = [(t, ro.rounded(t, e, dt)) for t, e in zip(grads, errs)]
    if table is not None:
        out.append((dtable, ro.rounded(dtable, et + ro.gamma(n + 300) * mt, dt)))
    return out
