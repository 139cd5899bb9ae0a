"""Group norm of samples in several pieces: values that are not finite, first rows far off, as many channels as are taken."""
import math

import pytest
import torch

import _mixing as mx
import _rowops as ro
import submanifold_sparse_convolution_amd as smc
from test_gpu_group_norm import BF16, F16, device_offsets, inputs

pytestmark = pytest.mark.gpu


# sample 1 has 40 rows of a piece, then pieces of 128: the first row and a later one of each; a norm of one launch
@pytest.mark.parametrize("row,off", [(r, [0, 40, 900, 1000]) for r in (40, 77, 128, 300, 899)]
                         + [(r, [0, 4, 9, 12]) for r in (4, 6, 8)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name,dt", [(None, BF16), ("relu", BF16), ("relu", F16)])
def test_values_that_are_not_finite_reach_their_sample_and_group(row, off, bad, name, dt):
    n, c, groups, (_, begin, end, _) = off[-1], 128, 16, off
    x, w, b, _ = (t.cuda() for t in inputs(n, c, dt, 31))
    o = device_offsets(off)
    y, stats = smc.group_norm(x, w, b, groups, offsets=o, activation=name, stats=True)
    x[row, 9] = bad
    got, stats2 = smc.group_norm(x, w, b, groups, offsets=o, activation=name, stats=True)
    assert torch.isnan(got[begin:end, 8:16]).all() and torch.isnan(stats2[1, 1, 1])
    got[begin:end, 8:16] = y[begin:end, 8:16]
    stats2[1, 1] = stats[1, 1]
    assert torch.equal(got, y) and torch.equal(stats2, stats)


# ---- variances of samples whose first rows lie far from the others ----------------------


def links(rows, n, c, groups):
    """(rows of a piece, most additions that follow each other on the way to a variance): rows of a thread,
    threads of a block, channels of a group, pieces of a sample."""
    words = -(-c // 8)
    lanes = 512 // words
    piece = -(-max(-(-n // 512), 4 * 512 // words) // lanes) * lanes
    pieces, parts = rows // piece + 2, 512 // groups
    return piece, (-(-piece // lanes) + math.ceil(math.log2(lanes)) + -(-(c // groups) // 64) + 6
                   + -(-pieces // parts) + math.ceil(math.log2(parts)) + 8)


# the sample begins one row before a cut of the rows into pieces (of 256 and 2,048 rows), and at a cut
@pytest.mark.parametrize("start", [2047, 2048])
@pytest.mark.parametrize("n,c,groups", [(91000, 64, 8), (1000000, 16, 2)])
@pytest.mark.parametrize("mean,first,dt", [(0, 100, BF16), (0, 1000, BF16), (0, 10000, F16), (300, 0, F16), (1000, 0, F16),
                                           (-1000, 1000, F16)])
def test_variance_with_a_first_row_far_off(start, n, c, groups, mean, first, dt):
    """The first row of the sample is `first`, the others are spread by 1 around `mean`.

    Bound. A running mean is at most `far` from its origin (a row of the piece, or a piece's mean) and rounds
    by u far at each of K additions, so a deviation errs by K u far, its square by 2 K u far |deviation|.
    Over a piece of R rows with its origin D off that is 2 K u D sum |deviations|, over all pieces at most
    2 K u sqrt(sum D^2) sqrt(R sum deviations^2), and each D^2 is part of the variance: 2 K u sqrt(R) of the
    variance, beside K u for the additions. rstd's relative error is half of the variance's, and 4 u."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    x = (torch.randn(n, c, generator=g, device="cuda") + mean).to(dt)
    x[start] = first
    w, b = torch.ones(c, dtype=dt, device="cuda"), torch.zeros(c, dtype=dt, device="cuda")
    _, stats = smc.group_norm(x, w, b, groups, offsets=device_offsets([0, start, n]), stats=True)
    v = x[start:].double().view(n - start, groups, -1)
    var, at = torch.var_mean(v, (0, 2), unbiased=False)
    rstd = (var + 1e-5) ** -0.5
    piece, k = links(n - start, n, c, groups)
    rel = 0.5 * ro.gamma(k) * (1 + 2 * math.sqrt(piece)) + 4 * ro.U
    assert ((stats[1, :, 1].double() - rstd).abs() <= rel * rstd).all(), ((stats[1, :, 1].double() / rstd - 1).abs().max(), rel)
    far = v.amax((0, 2)) - v.amin((0, 2))
    assert ((stats[1, :, 0].double() - at).abs() <= ro.gamma(k + 8) * far + 2 * ro.U * at.abs()).all()


@pytest.mark.parametrize("n", [16, 1000])
@pytest.mark.parametrize("row", [0, 7, 700])
def test_squares_past_float32(n, row):
    """A value whose square is no float32 number: the variance is infinite, x_hat 0 and y the bias."""
    x, w, b, _ = inputs(n, 128, BF16, 32)
    x[row % n, 5] = 2.0 ** 100
    y, stats = smc.group_norm(x.cuda(), w.cuda(), b.cuda(), 128, stats=True)
    assert stats[0, 5, 1] == 0 and torch.equal(y[:, 5].cpu(), b[5].expand(n))
    assert torch.isfinite(stats).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("n", [2, 5])
def test_as_many_channels_and_groups_as_are_taken(n):
    x, w, b, dy = inputs(n, 8192, BF16, 33)
    d = [t.double() for t in (x, w, b)]
    y, stats = smc.group_norm(x.cuda(), w.cuda(), b.cuda(), 4096, activation="silu", stats=True)
    ro.check(y, *mx.group_norm(*d, 4096, None, 1e-5, "silu", BF16), "y")
    got = smc.group_norm_backward(dy.cuda(), x.cuda(), w.cuda(), b.cuda(), 4096, stats, activation="silu")
    for t, (want, bound), label in zip(got, mx.group_norm_backward(dy.double(), *d, 4096, stats.double().cpu(), None, "silu", BF16),
                                       ("dx", "dw", "db")):
        ro.check(t, want, bound, label)
