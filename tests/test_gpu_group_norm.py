"""Group norm against its formulas in 64 bits, within the bounds of _mixing."""
import ctypes

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


def device_offsets(offsets):
    return None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")


def inputs(n, c, dt, seed):
    """x with a mean and a spread of its own in every channel."""
    g = gen(seed)
    x = (torch.randn(n, c, generator=g) * (0.5 + torch.rand(c, generator=g)) + torch.randn(c, generator=g)).to(dt)
    return x, normal(g, (c,), 0.3, dt) + 1, normal(g, (c,), 0.3, dt), normal(g, (n, c), 0.2, dt)


# (n, c, groups, offsets): one row, one channel, groups inside and across words, rows that are no
# whole words, samples without rows, rows of no sample, several pieces a sample and samples a piece
SHAPES = [
    (1, 512, 32, None), (1, 1, 1, None), (3, 8, 8, [0, 1, 3]), (27, 16, 4, None), (300, 33, 3, [0, 0, 100, 100, 300]),
    (257, 24, 8, [5, 60, 200]), (1000, 200, 10, [0, 1, 2, 700, 1000]), (5000, 7, 7, None), (4097, 64, 64, [0, 4096, 4097]),
    (9001, 128, 16, [0, 2000, 2001, 9000]), (3000, 512, 1, [0, 1500, 3000]), (40, 8192, 32, [0, 17, 40]),
    (70, 6000, 1000, None), (9, 4095, 4095, [2, 9]), (30000, 136, 17, [3, 3, 29000, 29000]),
    (700, 40, 5, list(range(0, 701, 7))), (200, 96, 12, [0] * 70 + list(range(0, 201, 2))),
]


@pytest.mark.parametrize("n,c,groups,offsets", SHAPES)
@pytest.mark.parametrize("name,dt", [(None, BF16), ("silu", BF16), ("gelu", F16), ("relu", F16)])
def test_forward(n, c, groups, offsets, name, dt):
    x, w, b, _ = inputs(n, c, dt, n + c)
    y, stats = smc.group_norm(x.cuda(), w.cuda(), b.cuda(), groups, offsets=device_offsets(offsets), activation=name, stats=True)
    d = [t.double() for t in (x, w, b)]
    ro.check(y, *mx.group_norm(*d, groups, offsets, 1e-5, name, dt), "y")
    mean, rstd, em, er = mx.group_stats(d[0], groups, offsets, 1e-5)
    ro.check(stats[:, :, 0], mean, em, "mean")
    ro.check(stats[:, :, 1], rstd, rstd * er, "rstd")
    again = smc.group_norm(x.cuda(), w.cuda(), b.cuda(), groups, offsets=device_offsets(offsets), activation=name)
    assert torch.equal(again, y)


@pytest.mark.parametrize("n,c,groups,offsets", SHAPES)
@pytest.mark.parametrize("name,dt", [(None, F16), ("silu", F16), ("gelu", BF16), ("relu", BF16)])
def test_backward(n, c, groups, offsets, name, dt):
    x, w, b, dy = inputs(n, c, dt, n + 2 * c)
    d = [t.double() for t in (x, w, b)]
    mean, rstd = mx.group_stats(d[0], groups, offsets, 1e-5)[:2]
    stats = torch.stack((mean, rstd), 2).float()
    if name == "relu":                      # the slope jumps at 0: nothing comes from there
        z = (d[0] - mx.spread(stats[:, :, 0].double(), d[0], offsets, groups)) * mx.spread(stats[:, :, 1].double(), d[0], offsets, groups)
        dy = torch.where((z * d[1] + d[2]).abs() < 1e-4, torch.zeros_like(dy), dy)
    got = smc.group_norm_backward(dy.cuda(), x.cuda(), w.cuda(), b.cuda(), groups, stats.cuda(),
                                  offsets=device_offsets(offsets), activation=name)
    want = mx.group_norm_backward(dy.double(), *d, groups, stats.double(), offsets, name, dt)
    for v, (wv, bound), label in zip(got, want, ("dx", "dweight", "dbias")):
        ro.check(v, wv, bound, label)


@pytest.mark.parametrize("name", [None, "silu", "gelu"])
def test_gradients_against_differences(name):
    """The formulas of _mixing (which the kernels are held to) against central
    differences of the forward formula in 64 bits; the kernels' own gradient, from
    their own statistics, along a random direction."""
    n, c, groups, offsets = 60, 12, 3, [2, 30, 30, 58]
    x, w, b, dy = inputs(n, c, F16, 5)
    d = [t.double() for t in (x, w, b)]

    def value(x, w, b):
        return (mx.group_norm(x, w, b, groups, offsets, 1e-5, name, F16)[0] * dy.double()).sum()

    mean, rstd = mx.group_stats(d[0], groups, offsets, 1e-5)[:2]
    want = [v for v, _ in mx.group_norm_backward(dy.double(), *d, groups, torch.stack((mean, rstd), 2), offsets, name, F16)]
    off = device_offsets(offsets)
    _, stats = smc.group_norm(x.cuda(), w.cuda(), b.cuda(), groups, offsets=off, activation=name, stats=True)
    got = smc.group_norm_backward(dy.cuda(), x.cuda(), w.cuda(), b.cuda(), groups, stats, offsets=off, activation=name)
    g = gen(8)
    for k in range(3):
        t = torch.randn(d[k].shape, generator=g, dtype=torch.float64)
        h = 1e-4
        hi, lo = ([v + s * h * t if i == k else v for i, v in enumerate(d)] for s in (1, -1))
        slope = (value(*hi) - value(*lo)) / (2 * h)
        # the third derivative's part: h^2 times values of order 10 |t|^3
        assert abs(slope - (want[k] * t).sum()) <= 1e-5 * (want[k] * t).abs().sum() + 1e-5
        # half an ulp of f16 an element, and as much again for what float32 leaves of the sums
        assert abs((got[k].double().cpu() * t).sum() - slope) <= 2.0 ** -10 * (want[k] * t).abs().sum() + 1e-5


def test_large_means_keep_their_variance():
    """Channels around 1,000 with a spread of a few units (whole numbers: exact in
    bf16 up to 256, so f16): float32 sums of squares would lose the variance."""
    g = gen(1)
    x = (1000 + torch.randint(-4, 5, (20000, 64), generator=g)).to(F16)
    w, b = torch.ones(64, dtype=F16), torch.zeros(64, dtype=F16)
    _, stats = smc.group_norm(x.cuda(), w.cuda(), b.cuda(), 4, stats=True)
    v = x.double().view(20000, 4, 16)
    var, mean = torch.var_mean(v, (0, 2), unbiased=False)
    # the sums are of whole numbers below 2^24, exact; means round a few times
    assert torch.allclose(stats[0, :, 0].double().cpu(), mean, rtol=4 * 2.0 ** -24, atol=0)
    assert torch.allclose(stats[0, :, 1].double().cpu(), (var + 1e-5) ** -0.5, rtol=1e-5, atol=0)


@pytest.mark.parametrize("extra,step", [(3, 1), (8, 1), (8, 2), (5, 3)])
def test_strided_rows(extra, step):
    n, c, groups, off = 500, 40, 5, [0, 123, 500]
    x, w, b, dy = inputs(n, c, BF16, 7)
    wide = torch.full((n * step, c + extra), float("nan"), dtype=BF16, device="cuda")
    xs, dys = wide[::step, extra:], wide.clone()[::step, extra:]
    xs.copy_(x)
    dys.copy_(dy)
    ws, bs = torch.cat((w[:1], w)).cuda()[1:], torch.cat((b[:1], b)).cuda()[1:]
    o = device_offsets(off)
    y, stats = smc.group_norm(x.cuda(), w.cuda(), b.cuda(), groups, offsets=o, activation="silu", stats=True)
    ys, stats_s = smc.group_norm(xs, ws, bs, groups, offsets=o, activation="silu", stats=True)
    assert torch.equal(y, ys) and torch.equal(stats, stats_s)
    grads = smc.group_norm_backward(dy.cuda(), x.cuda(), w.cuda(), b.cuda(), groups, stats, offsets=o, activation="silu")
    again = smc.group_norm_backward(dys, xs, ws, bs, groups, stats, offsets=o, activation="silu")
    assert all(torch.equal(p, q) for p, q in zip(grads, again))


def test_no_rows_and_constant_samples():
    w, b = torch.ones(16, dtype=BF16, device="cuda"), torch.full((16,), 2.0, dtype=BF16, device="cuda")
    none = torch.empty(0, 16, dtype=BF16, device="cuda")
    y, stats = smc.group_norm(none, w, b, 4, stats=True)
    assert y.shape == (0, 16) and torch.all(stats == 0)
    dx, dw, db = smc.group_norm_backward(none, none, w, b, 4, stats)
    assert dx.shape == (0, 16) and torch.all(dw == 0) and torch.all(db == 0)
    # no variance: x_hat is 0, with and without an epsilon, and so is dx
    x = torch.full((40, 16), 3.0, dtype=BF16, device="cuda")
    for eps in (1e-5, 0.0):
        y, stats = smc.group_norm(x, w, b, 4, eps=eps, stats=True)
        assert torch.all(y == 2) and torch.all(stats[:, :, 0] == 3)
        assert torch.all(torch.isfinite(stats))
    assert torch.all(stats[:, :, 1] == 0)


@pytest.mark.parametrize("name", [None, "silu", "gelu", "relu"])
def test_one_element_has_no_gradient(name):
    """A sample and group of one element: y does not depend on x."""
    x, w, b, dy = (t.cuda() for t in inputs(2, 24, BF16, 3))
    o = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    y, stats = smc.group_norm(x, w, b, 24, offsets=o, activation=name, stats=True)
    dx, _, _ = smc.group_norm_backward(dy, x, w, b, 24, stats, offsets=o, activation=name)
    assert torch.all(dx == 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_samples_do_not_reach_each_other(bad):
    """A value that is not finite stays in its sample (and, in dw and db, its group's channels)."""
    n, c, groups, off = 900, 32, 4, [0, 300, 301, 900]
    x, w, b, dy = (t.cuda() for t in inputs(n, c, BF16, 9))
    o = device_offsets(off)
    y, stats = smc.group_norm(x, w, b, groups, offsets=o, stats=True)
    grads = smc.group_norm_backward(dy, x, w, b, groups, stats, offsets=o)
    x[300, 9] = bad
    y2, stats2 = smc.group_norm(x, w, b, groups, offsets=o, stats=True)
    grads2 = smc.group_norm_backward(dy, x, w, b, groups, stats2, offsets=o)
    rows = torch.arange(n) != 300
    assert torch.equal(y[rows], y2[rows]) and torch.equal(stats[[0, 2]], stats2[[0, 2]])
    assert torch.equal(grads[0][rows], grads2[0][rows])
    assert not torch.isfinite(y2[300, 8:16]).any() and torch.equal(y[300, 16:], y2[300, 16:])
    others = torch.arange(c) // 8 != 1
    assert all(torch.equal(p[others], q[others]) for p, q in zip(grads[1:], grads2[1:]))


def test_in_place_and_refusals():
    n, c = 300, 64
    x, w, b, dy = (t.cuda() for t in inputs(n, c, BF16, 4))
    y, stats = smc.group_norm(x, w, b, 8, stats=True)
    dx, _, _ = smc.group_norm_backward(dy, x, w, b, 8, stats)
    L = smc.lib()
    a = smc._group_args(x, w, b, 8, None, 1e-5, None)
    ws = torch.empty(max(L.smc_group_norm_workspace(a), L.smc_group_norm_backward_workspace(a)), dtype=torch.uint8, device="cuda")
    xi = x.clone()
    a.x = a.y = xi.data_ptr()
    a.ldy, a.workspace, a.workspace_bytes = c, ws.data_ptr(), ws.numel()
    assert L.smc_group_norm(ctypes.byref(a), smc._raw_stream(x.device)) == 0
    assert torch.equal(xi, y)
    for over in ("x", "dy"):
        t = {"x": x.clone(), "dy": dy.clone()}
        dw, db = torch.empty_like(w), torch.empty_like(b)
        a.x, a.dy, a.ld_dy, a.dx, a.ld_dx = t["x"].data_ptr(), t["dy"].data_ptr(), c, t[over].data_ptr(), c
        a.dweight, a.dbias, a.stats = dw.data_ptr(), db.data_ptr(), stats.data_ptr()
        assert L.smc_group_norm_backward(ctypes.byref(a), smc._raw_stream(x.device)) == 0
        assert torch.equal(t[over], dx), over
    with pytest.raises(ValueError):
        smc.group_norm(x, w, b, 7)
    with pytest.raises(ValueError):
        smc.group_norm(x, w, b, 8, offsets=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        smc.group_norm(x, w, b, 8, offsets=torch.tensor([0, 300], device="cuda"))
    with pytest.raises(TypeError):
        smc.group_norm(x, w.half(), b, 8)
    with pytest.raises(ValueError):
        smc.group_norm(x, w, b, 8, activation="tanh")
    with pytest.raises(smc.SmconvError):
        smc.group_norm(x, w, b, 8, eps=-1.0)
    for c2, groups in ((4099, 4099), (8200, 8)):           # more groups, channels than a block holds
        v = torch.zeros(c2, dtype=BF16, device="cuda")
        with pytest.raises(smc.SmconvError, match="more than"):
            smc.group_norm(v.expand(2, c2).contiguous(), v, v, groups)
    with pytest.raises(ValueError):
        smc.group_norm_backward(dy, x, w, b, 8, stats[:, :4])
    with pytest.raises(ValueError):
        smc.group_norm_backward(dy[:5], x, w, b, 8, stats)


def test_streams_and_graph():
    """On another stream, and captured with both passes: replays on new inputs and
    other offsets give the eager bits."""
    n, c, groups = 5000, 64, 8
    x, w, b, dy = (t.cuda() for t in inputs(n, c, BF16, 12))
    o = device_offsets([0, 1000, 5000])
    side = torch.cuda.Stream()
    want = smc.group_norm(x, w, b, groups, offsets=o, activation="silu")
    side.wait_stream(torch.cuda.current_stream())
    got = smc.group_norm(x, w, b, groups, offsets=o, activation="silu", stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, stats = smc.group_norm(x, w, b, groups, offsets=o, activation="silu", stats=True)
        grads = smc.group_norm_backward(dy, x, w, b, groups, stats, offsets=o, activation="silu")
    for k in range(4):
        fresh = inputs(n, c, BF16, 20 + k)
        cuts = [[0, 1000, 5000], [0, 0, 5000], [7, 4000, 4001], [0, 5000, 5000]][k]
        x.copy_(fresh[0])
        dy.copy_(fresh[3])
        o.copy_(torch.tensor(cuts))
        ye, se = smc.group_norm(x, w, b, groups, offsets=o, activation="silu", stats=True)
        ge = smc.group_norm_backward(dy, x, w, b, groups, se, offsets=o, activation="silu")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ye) and torch.equal(stats, se) and all(torch.equal(p, q) for p, q in zip(grads, ge))
