"""Window attention: rows that belong to no window may hold anything."""
import math

import pytest
import torch

import submanifold_sparse_convolution_amd as smc
from test_gpu_attention import BF16, F16, Case

pytestmark = pytest.mark.gpu


# short, mid and long blocks, and rows that are no whole 16-byte words
@pytest.mark.parametrize("lengths,dim", [([20, 33, 9, 2, 1], 32), ([64, 130, 40], 32), ([500] * 16, 32), ([300, 40], 128),
                                         ([70, 9, 65], 33)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("cells", [False, True])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_rows_of_no_window_may_hold_anything(lengths, dim, bad, cells, dt):
    """q, k, v and dout that are not finite in rows before and after the windows: zeros there, and the bits of every
    other row and of the table's gradient stay."""
    c = Case(lengths, heads=4, kv=2, dim=dim, dt=dt, extent=(8, 8, 8) if cells else None, reach=3, before=70, after=150, seed=20)
    q, k, v, table = (t if t is None else t.contiguous() for t in c.device())
    dout = c.dout.cuda()
    outside = torch.ones(c.n, dtype=torch.bool, device="cuda")
    outside[c.order[c.offsets[0]:c.offsets[-1]].long().cuda()] = False

    def run():
        out, lse = smc.window_attention(q, k, v, c.windows, 4, bias=table, lse=True)
        return (out, lse, *smc.window_attention_backward(dout, q, k, v, out, lse, c.windows, 4, bias=table))

    want = run()
    for t in (q, k, v, dout):
        t[outside] = bad
    for label, a, b in zip(("out", "lse", "dq", "dk", "dv", "dbias"), run(), want):
        if a is not None:
            assert torch.equal(a, b), label
    assert all((t[outside] == 0).all() for t in (want[0], *want[2:5]))
