"""Window attention at its edges: the sides of the rules that pick its blocks, layouts,
masks and values that are not finite, streams and graphs, refusals."""
import ctypes
import math

import pytest
import torch

import _mixing as mx
import _rowops as ro
import submanifold_sparse_convolution_amd as smc
from test_gpu_attention import BF16, F16, Case, backward, gen, normal

pytestmark = pytest.mark.gpu


def both(c):
    """Forward and backward of a case within the bounds of the formulas."""
    q, k, v, table = c.device()
    out, lse = smc.window_attention(q, k, v, c.windows, c.heads, bias=table, lse=True)
    want, bound, wl, el = mx.attention(*c.formula())
    ro.check(out, want, bound, "out")
    inside = ~torch.isinf(wl)
    ro.check(lse.cpu()[inside], wl[inside], el[inside], "lse")
    for t, (w, b), label in zip(backward(c, q, k, v, table), mx.attention_backward(c.dout.double(), *c.formula()),
                                ("dq", "dk", "dv", "dbias")):
        ro.check(t, w, b, label)


# Long blocks: rows mostly in long windows, and as many blocks of 128 rows as there are compute units; two heads a
# block where there are 16 blocks a unit; short blocks below 40 rows a window on average, whatever the longest
BLOCKS = {
    "long": dict(lengths=[500] * 16, heads=4, kv=4, dim=32),
    "long cells": dict(lengths=[500, 513] * 8, heads=4, kv=2, dim=32, extent=(32, 16, 16), reach=7),
    "long wide": dict(lengths=[640, 130] * 5, heads=8, kv=8, dim=64, extent=(8, 8, 8)),
    "long wide f16": dict(lengths=[700] * 11, heads=4, kv=2, dim=100, dt=F16, extent=(40, 40, 4), reach=9),
    "long f16": dict(lengths=[385] * 20, heads=4, kv=1, dim=64, dt=F16),
    "two long heads": dict(lengths=[200] * 270, heads=8, kv=4, dim=16),
    "two heads and one": dict(lengths=[20, 70, 41] * 160, heads=5, kv=1, dim=16, extent=(4, 4, 4)),
    "two short heads": dict(lengths=[9, 33, 4, 64, 65] * 160, heads=7, kv=7, dim=16, dt=F16, extent=(5, 8, 3), reach=2),
    "short and one of 300": dict(lengths=[2] * 2000 + [300], heads=2, kv=1, dim=32, extent=(10, 4, 10), reach=5),
    "rows alone and one of 900": dict(lengths=[2] * 300 + [900], heads=2, kv=2, dim=40, extent=(10, 10, 10), reach=5),
}


@pytest.mark.parametrize("name", BLOCKS)
def test_blocks(name):
    both(Case(**BLOCKS[name]))


# ---- layouts -----------------------------------------------------------------------


@pytest.mark.parametrize("dim,extent,first,extra", [(32, (6, 6, 6), 1, 3), (64, None, 8, 8), (33, (9, 9, 2), 0, 1),
                                                    (24, None, 3, 0)])
def test_rows_at_any_distance(dim, extent, first, extra):
    """Rows of one buffer, gradients into the columns of another and out into a third, none of them at
    16-byte words but in the second; what lies beside them stays."""
    c = Case([70, 5, 130], heads=4, kv=2, dim=dim, extent=extent, before=3, after=4, seed=5)
    wide = c.qkv.shape[1]
    buf = torch.full((c.n, first + wide + extra), 9.0, dtype=BF16, device="cuda")
    buf[:, first:first + wide] = c.qkv.cuda()
    q, k, v = buf[:, first:first + wide].split((4 * dim, 2 * dim, 2 * dim), 1)
    table = None if c.table is None else c.table.cuda()
    want, bound, _, _ = mx.attention(*c.formula())
    room = torch.full((c.n, 4 * dim + first + extra), 7.0, dtype=BF16, device="cuda")
    out = room[:, first:first + 4 * dim]
    got, lse = smc.window_attention(q, k, v, c.windows, 4, bias=table, lse=True, out=out)
    assert got.data_ptr() == out.data_ptr()
    ro.check(got, want, bound, "out")
    assert (room[:, :first] == 7).all() and (room[:, first + 4 * dim:] == 7).all()
    grads = torch.full_like(buf, 5.0)
    dq, dk, dv = grads[:, first:first + wide].split((4 * dim, 2 * dim, 2 * dim), 1)
    dout = torch.full((c.n, 4 * dim + 2 * first), 3.0, dtype=BF16, device="cuda")
    dout[:, first:first + 4 * dim] = c.dout.cuda()
    _, _, _, dt = smc.window_attention_backward(dout[:, first:first + 4 * dim], q, k, v, want.to(BF16).cuda(), lse, c.windows,
                                                4, bias=table, grads=(dq, dk, dv))
    for t, (w, b), label in zip((dq, dk, dv, dt), mx.attention_backward(c.dout.double(), *c.formula()),
                                ("dq", "dk", "dv", "dbias")):
        ro.check(t, w, b, label)
    assert (grads[:, :first] == 5).all() and (grads[:, first + wide:] == 5).all()


def test_rows_past_32_bit_offsets():
    """Rows 2^16 elements apart: 5 GB of them, offsets beyond 2^32 bytes."""
    c = Case([40000 // 125] * 125, heads=2, kv=2, dim=16, seed=6)
    q, k, v, _ = c.device()
    want, lse = smc.window_attention(q, k, v, c.windows, 2, lse=True)
    gw = smc.window_attention_backward(c.dout.cuda(), q, k, v, want, lse, c.windows, 2)
    buf = torch.empty(c.n, 1 << 16, dtype=BF16, device="cuda")
    far = [buf[:, 32 * i:32 * i + 32] for i in (0, 1, 2, 2000, 2001, 2002, 3, 4)]
    for to, t in zip(far, (q, k, v)):
        to.copy_(t)
    far[7].copy_(c.dout.cuda())
    out = smc.window_attention(far[0], far[1], far[2], c.windows, 2, out=far[6])
    assert torch.equal(out, want)
    got = smc.window_attention_backward(far[7], far[0], far[1], far[2], out, lse, c.windows, 2, grads=far[3:6])
    assert all(torch.equal(a, b) for a, b in zip(got[:3], gw[:3]))


def test_scale_and_coordinates():
    """A scale of one's own; [N, 3] coordinates, anywhere in 32 bits, are [N, 4]'s."""
    c = Case([90, 31, 200], heads=4, kv=4, dim=16, extent=(12, 10, 9), reach=3, order=False, seed=7)
    q, k, v, table = c.device()
    out = smc.window_attention(q, k, v, c.windows, 4, bias=table, scale=0.71)
    args = list(c.formula())
    args[9] = 0.71
    want, bound, _, _ = mx.attention(*args)
    ro.check(out, want, bound, "out")
    o = torch.tensor(c.offsets, dtype=torch.int32, device="cuda")
    cells = c.coords[:, 1:] - c.coords[:, 1:].amin(0)       # the first window's lowest, not every one's
    for edge in (-2 ** 31, 2 ** 31 - 1 - int(cells.max())):
        w = smc.Windows(o, c.n, coords=(cells.long() + edge).int().cuda(), extent=(12, 10, 9))
        assert torch.equal(smc.window_attention(q, k, v, w, 4, bias=table, scale=0.71), out)
    far = torch.zeros(2, 3, dtype=torch.int32)
    far[0], far[1] = -2 ** 31, 2 ** 31 - 1
    with pytest.raises(smc.SmconvError, match="extent"):
        smc.Windows(torch.tensor([0, 2], dtype=torch.int32, device="cuda"), 2, coords=far.cuda(), extent=(4, 4, 4))


# ---- masks and values that are not finite -------------------------------------------


def masked(c, entries, value):
    for axis, bucket, head in entries:
        c.table[axis, bucket, head] = value
    return c.table.cuda()


def counted(c):
    """The table as it counts: entries of at most 2^14."""
    table = c.table
    c.table = table.float().clamp(-2.0 ** 14, 2.0 ** 14).to(c.dt)
    args = c.formula()
    c.table = table
    return args


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("value", ["-inf", "lowest", "-1e5", "inf"])
@pytest.mark.parametrize("length", [50, 300])
def test_masks_in_the_table(dt, value, length):
    """Infinite and lowest entries: keys without a share; one of head 1's is the distance zero, so that
    cells alone in their window's corner have only masked keys; every entry of head 2 is masked."""
    c = Case([length, 7, 1, 64], heads=3, kv=3, dim=32, dt=dt, extent=(6, 5, 9), reach=2, seed=8)
    number = {"-inf": -math.inf, "lowest": torch.finfo(dt).min, "-1e5": max(-1e5, torch.finfo(dt).min), "inf": math.inf}[value]
    entries = [(0, 0, 0), (1, 3, 0), (0, 2, 1)] + [(a, b, 2) for a in range(3) for b in range(5)]
    table = masked(c, entries, number)
    q, k, v, _ = c.device()
    args = counted(c)
    want, bound, wl, el = mx.attention(*args)
    out, lse = smc.window_attention(q, k, v, c.windows, 3, bias=table, lse=True)
    ro.check(out, want, bound, "out")
    ro.check(lse, wl, el, "lse")
    got = smc.window_attention_backward(c.dout.cuda(), q, k, v, want.to(dt).cuda(), wl.float().cuda(), c.windows, 3, bias=table)
    for t, (w, b), label in zip(got, mx.attention_backward(c.dout.double(), *args), ("dq", "dk", "dv", "dbias")):
        ro.check(t, w, b, label)


@pytest.mark.parametrize("length", [30, 200])
def test_rows_whose_scores_are_all_minus_infinity(length):
    """q k overflows float32: zeros, lse -inf, and no gradient; the other rows do not change."""
    c = Case([length, 40], heads=2, kv=2, dim=32, order=False, seed=9)
    c.k[:length, 0] = c.k[:length, 0].abs() + 1
    q, k, v, _ = c.device()
    want, wl = smc.window_attention(q, k, v, c.windows, 2, lse=True)
    gw = smc.window_attention_backward(c.dout.cuda(), q, k, v, want, wl, c.windows, 2)
    q2 = q.clone()
    q2[3, 0] = -math.inf
    out, lse = smc.window_attention(q2, k, v, c.windows, 2, lse=True)
    assert (out[3, :32] == 0).all() and lse[0, 3] == -math.inf
    rows = torch.arange(c.n, device="cuda") != 3
    assert torch.equal(out[rows], want[rows]) and torch.equal(out[3, 32:], want[3, 32:]) and torch.equal(lse[:, rows], wl[:, rows])
    got = smc.window_attention_backward(c.dout.cuda(), q2, k, v, out, lse, c.windows, 2)
    assert torch.equal(got[0][rows], gw[0][rows]) and torch.equal(got[0][3, 32:], gw[0][3, 32:])
    for t, w in zip(got[1:3], gw[1:3]):                      # the other head and the other window
        assert torch.equal(t[:, 32:], w[:, 32:]) and torch.equal(t[length:], w[length:])
    assert torch.isfinite(got[2]).all()


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("lengths", [[20, 33, 9, 2, 1], [64, 130, 40], [500] * 16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_windows_do_not_reach_each_other(dt, lengths, bad):
    """A window of NaN or infinities in q, k, v and dout: the others' outputs and gradients keep their bits."""
    c = Case(lengths, heads=4, kv=2, dim=32, dt=dt, extent=(8, 8, 8), reach=3, before=5, after=6, seed=10)
    q, k, v, table = (t.contiguous() for t in c.device())
    dout = c.dout.cuda()
    out, lse = smc.window_attention(q, k, v, c.windows, 4, bias=table, lse=True)
    want = smc.window_attention_backward(dout, q, k, v, out, lse, c.windows, 4, bias=table)
    hit = c.order[c.offsets[1]:c.offsets[2]].long().cuda()
    rest = torch.ones(c.n, dtype=torch.bool, device="cuda")
    rest[hit] = False
    for t in (q, k, v, dout):
        t[hit] = bad
    out2, lse2 = smc.window_attention(q, k, v, c.windows, 4, bias=table, lse=True)
    got = smc.window_attention_backward(dout, q, k, v, out2, lse2, c.windows, 4, bias=table)
    assert torch.equal(out2[rest], out[rest]) and not torch.isfinite(out2[hit]).any()
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a[rest], b[rest])
    outside = torch.ones(c.n, dtype=torch.bool, device="cuda")
    outside[c.order[c.offsets[0]:c.offsets[-1]].long().cuda()] = False
    assert all((t[outside] == 0).all() for t in (out2, *got[:3]))


def test_windows_of_one_row_have_no_gradient():
    """P is 1 whatever q and k are: dq and dk exactly zero, dv is dout (summed over the heads that share v)."""
    for dt, kv in ((BF16, 4), (F16, 2)):
        c = Case([1] * 90, heads=4, kv=kv, dim=32, dt=dt, extent=(1, 1, 1), reach=1, seed=11)
        q, k, v, table = c.device()
        out, lse = smc.window_attention(q, k, v, c.windows, 4, bias=table, lse=True)
        assert torch.equal(out, v.reshape(90, kv, 1, 32).expand(90, kv, 4 // kv, 32).reshape(90, 128))
        dq, dk, dv, dbias = smc.window_attention_backward(c.dout.cuda(), q, k, v, out, lse, c.windows, 4, bias=table)
        assert (dq == 0).all() and (dk == 0).all() and (dbias == 0).all()
        assert torch.equal(dv.cpu(), c.dout.float().view(90, kv, 4 // kv, 32).sum(2).reshape(90, -1).to(dt))


def test_more_windows_than_a_grid_has_blocks():
    """70,000 windows of a row between 70,000 of none, with cells: out is v."""
    n = 70000
    g = gen(15)
    offsets = torch.arange(n + 1).repeat_interleave(2)[:-1].int().cuda()
    coords = torch.randint(-2 ** 20, 2 ** 20, (n, 3), generator=g).int().cuda()
    order = torch.randperm(n, generator=g).int().cuda()
    w = smc.Windows(offsets, n, order=order, coords=coords, extent=(1, 1, 1))
    q, k, v = (normal(g, (n, 64)).cuda() for _ in range(3))
    table = normal(g, (3, 3, 2)).cuda()
    out, lse = smc.window_attention(q, k, v, w, 2, bias=table, lse=True)
    assert w.longest == 1 and torch.equal(out, v)
    dout = normal(g, (n, 64)).cuda()
    dq, dk, dv, dbias = smc.window_attention_backward(dout, q, k, v, out, lse, w, 2, bias=table)
    assert torch.equal(dv, dout) and (dq == 0).all() and (dk == 0).all() and (dbias == 0).all()


@pytest.mark.parametrize("size", [2.0 ** -14, 1.0, 2.0 ** 12])
@pytest.mark.parametrize("lengths", [[20, 33, 9], [200, 64, 65]])
def test_f16_gradients_of_any_size(size, lengths):
    """dS is scaled window by window: small and large gradients within the bound, which follows their size."""
    c = Case(lengths, heads=2, kv=1, dim=32, dt=F16, extent=(6, 6, 6), seed=12)
    c.dout = (c.dout.float() * size).to(F16)
    q, k, v, table = c.device()
    for t, (w, b), label in zip(backward(c, q, k, v, table), mx.attention_backward(c.dout.double(), *c.formula()),
                                ("dq", "dk", "dv", "dbias")):
        ro.check(t, w, b, label)


# ---- streams, graphs, several calls ----------------------------------------------------


@pytest.mark.parametrize("dt", [BF16, F16])
def test_streams_and_graph(dt):
    """On another stream; two captured calls on the same windows, replayed on new inputs between eager calls."""
    c = Case([50, 64, 130, 7], heads=4, kv=2, dim=32, dt=dt, extent=(9, 9, 9), reach=4, seed=13)
    q, k, v, table = (t.contiguous() for t in c.device())
    dout = c.dout.cuda()

    def run(**kw):
        out, lse = smc.window_attention(q, k, v, c.windows, 4, bias=table, lse=True, **kw)
        return (out, lse, *smc.window_attention_backward(dout, q, k, v, out, lse, c.windows, 4, bias=table, **kw))

    def equal(a, b):
        return all(torch.equal(x, y) for x, y in zip(a, b))

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(stream=side)
    again = run()                                           # at the same time, on this one
    torch.cuda.synchronize()
    assert equal(got, want) and equal(again, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one = run()
        two = run()
    for i in range(4):
        fresh = Case([50, 64, 130, 7], heads=4, kv=2, dim=32, dt=dt, extent=(9, 9, 9), reach=4, seed=50 + i)
        for t, f in zip((q, k, v, table), fresh.device()):
            t.copy_(f)
        dout.copy_(fresh.dout.cuda() * 2.0 ** (3 * i))
        eager = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert equal(one, eager) and equal(two, eager)


def test_no_rows():
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    for offsets in (o, o[:1]):
        w = smc.Windows(offsets, 0, coords=torch.empty(0, 4, dtype=torch.int32, device="cuda"), extent=(4, 4, 4))
        assert w.longest == 0
        table = torch.zeros(3, 3, 2, dtype=BF16, device="cuda")
        out, lse = smc.window_attention(e, e, e, w, 2, bias=table, lse=True)
        assert out.shape == (0, 64) and lse.shape == (2, 0)
        dq, dk, dv, dbias = smc.window_attention_backward(e, e, e, e, out, lse, w, 2, bias=table)
        assert dq.shape == dk.shape == dv.shape == (0, 64) and (dbias == 0).all()


# ---- refusals ----------------------------------------------------------------------------


def device(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def test_windows_that_are_refused():
    """Bad offsets, orders and cells are found on the device; the same memory serves the next windows."""
    def status(*args, **kw):
        with pytest.raises(smc.SmconvError) as e:
            smc.Windows(*args, **kw)
        return e.value.status

    RANGE, DUPLICATE, UNSUPPORTED = 2, 3, 4
    assert status(device(0, 2, 4), 4, order=device(0, 1, 1, 3)) in (RANGE, DUPLICATE)
    dup = status(device(0, 2, 4), 4, order=device(0, 1, 1, 3))
    rng = status(device(0, 2, 4), 4, order=device(0, 1, 2, 4))
    assert dup != rng
    assert status(device(0, 2, 4), 4, order=device(0, -1, 2, 3)) == rng
    assert status(device(0, 3, 2, 4), 4) == rng
    assert status(device(0, 2, 5), 4) == rng
    assert status(device(-1, 2, 4), 4) == rng
    cells = torch.zeros(4, 4, dtype=torch.int32)
    cells[3, 2] = 5
    assert status(device(0, 2, 4), 4, coords=cells.cuda(), extent=(4, 5, 4)) == rng
    assert smc.Windows(device(0, 2, 4), 4, coords=cells.cuda(), extent=(4, 6, 4)).longest == 2
    assert smc.Windows(device(0, 3, 4), 4, coords=cells.cuda(), extent=(1, 1, 1)).longest == 3
    assert status(device(0, 2, 4), 4, coords=cells.cuda(), extent=(64, 64, 4)) not in (dup, rng)
    assert status(device(0, 2, 4), 4, coords=cells.cuda(), extent=(0, 4, 4)) not in (dup, rng)
    with pytest.raises(ValueError):
        smc.Windows(device(0, 4), 4, coords=cells.cuda())
    with pytest.raises(ValueError):
        smc.Windows(device(0, 4), 4, extent=(4, 4, 4))
    with pytest.raises(ValueError):
        smc.Windows(device(0, 4), 4, order=device(0, 1, 2))
    with pytest.raises(ValueError):
        smc.Windows(device(0, 4), 4, coords=cells[:3].cuda(), extent=(8, 8, 8))
    with pytest.raises(TypeError):
        smc.Windows(torch.tensor([0, 4]), 4)
    with pytest.raises(TypeError):
        smc.Windows(torch.tensor([0, 4], device="cuda"), 4)


def test_calls_that_are_refused():
    c = Case([20, 12], heads=4, kv=2, dim=16, extent=(4, 4, 4), reach=2, seed=14)
    q, k, v, table = c.device()
    w = c.windows

    def call(*args, heads=4, **kw):
        return smc.window_attention(*args, w, heads, **kw)

    for args, kw in (((q, k, v), dict(heads=5)), ((q, k[:, :20], v[:, :20]), {}), ((q, k, v[:, :16]), {}),
                     ((q[:31], k, v), {}), ((q, k[:31], v), {}), ((q, k, v), dict(bias=table[:2].contiguous())),
                     ((q, k, v), dict(bias=table[:, :4].contiguous())), ((q, k, v), dict(bias=table[..., :3].contiguous())),
                     ((q, k, v), dict(out=q.new_empty(32, 63)))):
        with pytest.raises(ValueError):
            call(*args, **kw)
    for args, kw in (((q, k.half(), v), {}), ((q.float(), k.float(), v.float()), {}), ((q, k, v), dict(bias=table.float()))):
        with pytest.raises(TypeError):
            call(*args, **kw)
    with pytest.raises(TypeError):
        smc.window_attention(q, k, v, device(0, 20, 32), 4)
    plain = smc.Windows(device(0, 20, 32), 32)
    with pytest.raises(ValueError, match="coords"):
        smc.window_attention(q, k, v, plain, 4, bias=table)
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(out=q),
               dict(bias=torch.zeros(3, 257, 4, dtype=BF16, device="cuda"))):
        with pytest.raises(smc.SmconvError):
            call(q, k, v, **kw)
    wide = torch.zeros(32, 4 * 129, dtype=BF16, device="cuda")
    with pytest.raises(smc.SmconvError, match="head_dim"):
        call(wide, wide, wide)
    out, lse = call(q, k, v, bias=table, lse=True)
    dout = c.dout.cuda()

    def back(out=out, lse=lse, dout=dout, **kw):
        return smc.window_attention_backward(dout, q, k, v, out, lse, w, 4, bias=table, **kw)

    for kw in (dict(lse=lse[:3]), dict(out=out[:31]), dict(dout=dout[:, :60])):
        with pytest.raises(ValueError):
            back(**kw)
    with pytest.raises(TypeError):
        back(lse=lse.double())
    dq, dk, dv = (torch.empty_like(t.contiguous()) for t in (q, k, v))
    for grads in ((dq, dk, dk), (q, dk, dv), (dq, k, dv), (dout, dk, dv), (out, dk, dv), (dq, dq[:, :32], dv)):
        with pytest.raises(smc.SmconvError, match="shares memory"):
            back(grads=grads)
    # a plan that was not built
    a = smc.AttentionArgs()
    made = smc.WindowsArgs()
    ctypes.memmove(ctypes.byref(made), ctypes.byref(w._args), ctypes.sizeof(made))
    made.tiles32 = made.tiles64 = made.tiles128 = 0
    a.windows, a.heads, a.kv_heads, a.head_dim, a.scale = ctypes.pointer(made), 4, 2, 16, 0.25
    a.q, a.ldq, a.k, a.ldk, a.v, a.ldv = q.data_ptr(), 128, k.data_ptr(), 128, v.data_ptr(), 128
    a.out, a.ld_out = out.data_ptr(), 64
    assert smc.lib().smc_window_attention(ctypes.byref(a), smc._raw_stream(q.device)) != 0
