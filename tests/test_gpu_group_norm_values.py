"""Group norm of samples in several pieces: values that are not finite, wherever they lie."""
import math

import pytest
import torch

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
