"""Window attention against its formulas in 64 bits, within the bounds of _mixing."""
import itertools

import pytest
import torch

import _mixing as mx
import _rowops as ro
import submanifold_sparse_convolution_amd as smc

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, shape, std=1.0, dt=BF16):
    return (torch.randn(shape, generator=g) * std).to(dt)


class Case:
    """Inputs of one call on the CPU and its windows on the GPU. lengths: of the windows;
    before, after: rows of no window; extent None: no bias."""

    def __init__(self, lengths, heads, kv, dim, dt=BF16, extent=None, reach=2, order=True, before=0, after=0, seed=0,
                 spread=0.7):
        g = gen(seed + 31 * len(lengths) + dim)
        self.offsets = [before] + [before + s for s in itertools.accumulate(lengths)]
        self.n = n = self.offsets[-1] + after
        self.heads, self.kv, self.dim, self.dt = heads, kv, dim, dt
        self.order = torch.randperm(n, generator=g).int() if order else None
        self.qkv = normal(g, (n, (heads + 2 * kv) * dim), 1.0, dt)
        self.q, self.k, self.v = self.qkv.split((heads * dim, kv * dim, kv * dim), 1)
        self.dout = normal(g, (n, heads * dim), 0.1, dt)
        self.coords = self.table = self.extent = None
        if extent is not None:
            self.extent = extent
            self.coords = torch.zeros(n, 4, dtype=torch.int32)
            for places, rows in mx.window_rows(self.offsets, self.order, n):
                cells = torch.stack([torch.randint(0, e, (len(rows),), generator=g) for e in extent], 1)
                self.coords[rows, 1:] = (cells + torch.randint(-500, 500, (3,), generator=g)).int()
            self.table = normal(g, (3, 2 * reach + 1, heads), spread, dt)
        self.windows = smc.Windows(torch.tensor(self.offsets, dtype=torch.int32, device="cuda"), n,
                                   order=None if self.order is None else self.order.cuda(),
                                   coords=None if extent is None else self.coords.cuda(), extent=extent)

    def device(self):
        q, k, v = self.qkv.cuda().split((self.heads * self.dim, self.kv * self.dim, self.kv * self.dim), 1)
        return q, k, v, None if self.table is None else self.table.cuda()

    def formula(self):
        """The arguments of _mixing's formulas."""
        cells = None if self.coords is None else self.coords[:, 1:].long()
        table = None if self.table is None else self.table.double()
        return (self.q.double(), self.k.double(), self.v.double(), self.offsets, self.order, cells, table,
                self.heads, self.kv, self.dim ** -0.5, self.dt)


# lengths on the sides of the tiles' borders, head sizes that are no multiple of anything, shared heads, one cell and
# 128 cells, rows of no window, windows of a row and of none
CASES = {
    "one row": dict(lengths=[1], heads=1, kv=1, dim=32),
    "rows alone": dict(lengths=[1] * 70, heads=2, kv=1, dim=16, extent=(1, 1, 1), reach=1),
    "three cells": dict(lengths=[27], heads=8, kv=8, dim=64, extent=(3, 3, 3), order=False),
    "empty windows": dict(lengths=[0, 5, 0, 0, 64, 65, 0], heads=2, kv=2, dim=32, before=7, after=70),
    "no windows": dict(lengths=[], heads=2, kv=2, dim=32, after=130),
    "borders": dict(lengths=[15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129], heads=2, kv=2, dim=32,
                    extent=(12, 12, 8), reach=11),
    "f16 borders": dict(lengths=[15, 16, 17, 63, 64, 65, 128, 129], heads=2, kv=1, dim=64, dt=F16,
                        extent=(20, 20, 20), reach=4),
    "odd dim": dict(lengths=[50, 100, 3], heads=3, kv=1, dim=33, extent=(5, 6, 7), reach=3),
    "dim 1": dict(lengths=[9, 70], heads=4, kv=2, dim=1, dt=F16),
    "dim 24": dict(lengths=[200, 40], heads=6, kv=2, dim=24, dt=F16, order=False),
    "dim 100": dict(lengths=[90, 200], heads=2, kv=2, dim=100, extent=(16, 8, 40)),
    "dim 128": dict(lengths=[300, 64], heads=2, kv=1, dim=128, extent=(100, 20, 8), reach=127),
    "dim 127": dict(lengths=[70], heads=1, kv=1, dim=127, dt=F16, extent=(2, 2, 2), reach=1),
    "long": dict(lengths=[1025], heads=2, kv=2, dim=64),
    "long with cells": dict(lengths=[1500, 700], heads=2, kv=2, dim=32, extent=(40, 40, 11), reach=15),
    "long f16": dict(lengths=[600, 600], heads=4, kv=2, dim=48, dt=F16, extent=(30, 30, 4), reach=6, order=False),
    "long dim 128": dict(lengths=[520, 513], heads=2, kv=2, dim=128, dt=F16, extent=(64, 32, 32), reach=31),
}


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    c = Case(**CASES[name])
    q, k, v, table = c.device()
    out, lse = smc.window_attention(q, k, v, c.windows, c.heads, bias=table, lse=True)
    want, bound, wl, el = mx.attention(*c.formula())
    ro.check(out, want, bound, "out")
    got, none = lse.double().cpu(), torch.isinf(wl)
    assert torch.equal(got[none], wl[none])
    ro.check(torch.where(none, torch.zeros_like(got), got), torch.where(none, torch.zeros_like(wl), wl), el, "lse")
    assert torch.equal(smc.window_attention(q, k, v, c.windows, c.heads, bias=table), out)


def backward(c, q, k, v, table, dout=None):
    """The kernels' gradients, from the formula's out and lse (rounded)."""
    want, _, lse, _ = mx.attention(*c.formula())
    dout = c.dout if dout is None else dout
    return smc.window_attention_backward(dout.cuda(), q, k, v, want.to(c.dt).cuda(), lse.float().cuda(), c.windows, c.heads,
                                         bias=table)


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    c = Case(**CASES[name])
    q, k, v, table = c.device()
    got = backward(c, q, k, v, table)
    want = mx.attention_backward(c.dout.double(), *c.formula())
    for t, (w, bound), label in zip(got, want, ("dq", "dk", "dv", "dbias")):
        ro.check(t, w, bound, label)
    assert (got[3] is None) == (table is None)
    again = backward(c, q, k, v, table)
    assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)
