"""Row operators at the edges of their contract: outputs over inputs, values at
the ends of the types, long row ranges, more rows than one launch's grid counts."""
import ctypes

import pytest
import torch

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


def stream():
    return smc._raw_stream(torch.device("cuda", torch.cuda.current_device()))


# ---- the norm's outputs over its inputs --------------------------------------------


def norm_call(x, w, residual=None, y=None, scale=None, s=None, eps=1e-6):
    """smc_rms_norm on the given buffers (rows may be strided)."""
    n, c = x.shape
    return smc.lib().smc_rms_norm(ctypes.byref(smc.NormArgs(
        n, c, 0 if x.dtype == BF16 else 1, eps, x.data_ptr(), x.stride(0),
        None if residual is None else residual.data_ptr(), 0 if residual is None else residual.stride(0),
        w.data_ptr(), y.data_ptr(), y.stride(0), None if scale is None else scale.data_ptr(),
        None if s is None else s.data_ptr(), 0 if s is None else s.stride(0))), stream())


# rows in a lane group's registers, in a wave's, and re-read by a block (c > 4096)
@pytest.mark.parametrize("n,c", [(700, 33), (700, 128), (300, 512), (90, 1000), (40, 4096), (40, 4104), (40, 4099)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_norm_over_its_inputs(n, c, e4m3):
    g = gen(n + c)
    x, r, w = (normal(g, (n, c), v).cuda() for v in (1.0, 2.0, 0.0))
    w += normal(g, (c,)).cuda()
    w = w[0].contiguous()
    y = torch.empty(n, c, dtype=ro.E4M3 if e4m3 else BF16, device="cuda")
    scale = torch.empty(n, device="cuda") if e4m3 else None
    s = torch.empty_like(x)
    assert norm_call(x, w, r, y, scale, s) == 0
    bits = y.view(torch.uint8 if e4m3 else torch.int16).clone()
    for over in ("s = x", "s = residual") + (() if e4m3 else ("y = x", "y = x, s = residual")):
        xi, ri, yi, si = x.clone(), r.clone(), torch.empty_like(y), torch.empty_like(s)
        ki = torch.empty_like(scale) if e4m3 else None
        if "s = x" in over:
            si = xi
        if "s = residual" in over:
            si = ri
        if "y = x" in over:
            yi = xi
        assert norm_call(xi, w, ri, yi, ki, si) == 0
        assert torch.equal(yi.view(bits.dtype), bits), over
        assert torch.equal(si, s), over
        if e4m3:
            assert torch.equal(ki, scale), over


def test_e4m3_norm_beside_its_input():
    """e4m3 rows in columns of the buffer that holds x: equal row distances in
    bytes, no byte shared."""
    g = gen(5)
    n, c = 300, 64
    buf = torch.zeros(n, 256, dtype=torch.uint8, device="cuda")
    x = buf.view(BF16)[:, :c]
    x.copy_(normal(g, (n, c)))
    y = buf[:, 2 * c:3 * c].view(ro.E4M3)
    w = torch.ones(c, dtype=BF16, device="cuda")
    scale = torch.empty(n, device="cuda")
    before = x.clone()
    assert norm_call(x, w, None, y, scale) == 0
    q, want = smc.rms_norm(before, w, e4m3=True)
    assert torch.equal(y.view(torch.uint8), q.view(torch.uint8)) and torch.equal(scale, want)
    assert torch.equal(x, before) and torch.all(buf[:, 3 * c:] == 0)


# ---- f16 gradients whose dz is outside f16 ------------------------------------------


def d(t):
    return None if t is None else t.double()


def f16_gradients(halves, dy, x, w, b, name):
    """dz and (dx, dw, db) in 64 bits with the bounds of _rowops, where the stored dz
    is within half an ulp of f16 and 2^-17 of its largest value: the smallest step
    of f16 is 2^-24, and a largest value below 2^-8 is scaled up first."""
    back = ro.linear_backward if halves == 1 else ro.gated_backward
    z, _ = ro.pre(d(x), d(w), d(b))
    if halves == 1:
        dz = d(dy) * ro.slope(z, name)
    else:
        f = dy.shape[1]
        dz = torch.cat((d(dy) * z[:, f:] * ro.slope(z[:, :f], name), d(dy) * ro.act(z[:, :f], name)), 1)
    floor = ro.FLOOR[F16]
    try:                                    # the rounding floor of dz: 2^-17 of the largest
        ro.FLOOR[F16] = float(dz.abs().max()) * 2.0 ** -17
        wide = back(d(dy), d(x), d(w), d(b), name, F16)
    finally:
        own = ro.FLOOR[F16]
        ro.FLOOR[F16] = floor
    return dz, [(v, bd - own + floor) for v, bd in wide]


# (rows, c_in, c_out): one tile, several, odd sizes, all tile shapes of the slopes
RANGE_SHAPES = [(1, 16, 24), (40, 72, 33), (300, 128, 96), (2500, 64, 200), (9000, 64, 264), (3000, 512, 520)]


@pytest.mark.parametrize("n,c_in,c_out", RANGE_SHAPES)
@pytest.mark.parametrize("name", ["silu", "gelu", None])
def test_f16_gradients_with_large_dz(n, c_in, c_out, name):
    """dh times the up half is up to 10^6 or so, small weights bring dx, dW and
    db back into f16."""
    g = gen(n + c_in)
    x = normal(g, (n, c_in), 0.02, F16)
    w = normal(g, (c_in, 2 * c_out), 2.0 ** -9 / n ** 0.5, F16)
    b = torch.cat((torch.full((c_out,), 2.0), torch.full((c_out,), 500.0))).to(F16)
    dh = (normal(g, (n, c_out), 0.02, F16).float() + 1).to(F16)
    dh[0, 0], dh[n // 2, c_out // 2] = 400.0, -300.0
    sign = torch.where(torch.rand(n, c_out, generator=g) < 0.5, -1.0, 1.0)
    dh = (dh.float() * sign / n ** 0.5).to(F16)
    dh[n - 1, c_out - 1] = 300.0            # times 500: 150,000 or so, beyond f16
    dz, want = f16_gradients(2, dh, x, w, b, name)
    assert dz.abs().max() > 65504 * 1.5
    assert all(v.abs().max() < 65504 for v, _ in want[:2])
    got = smc.gated_backward(dh.cuda(), x.cuda(), w.cuda(), bias=b.cuda(), activation=name)
    for v, (wv, bd), label in zip(got[:2], want[:2], ("dx", "dw")):
        assert torch.isfinite(v).all(), label
        ro.check(v, wv, bd, label)
    keep = want[2][0].abs() < 65000         # a column sum may itself be beyond f16
    ro.check(got[2][keep.cuda()], want[2][0][keep], want[2][1][keep], "db")
    assert keep.sum() >= c_out


@pytest.mark.parametrize("n,c_in,c_out", RANGE_SHAPES)
@pytest.mark.parametrize("halves", [1, 2])
def test_f16_gradients_with_small_dz(n, c_in, c_out, halves):
    """A loss that nobody scaled: every dz is below f16's normal range, the
    gradients of the weights (x of 2,000) and of x (weights of 30) are not."""
    g = gen(n + c_in + halves)
    x = normal(g, (n, c_in), 2000.0, F16)
    w = normal(g, (c_in, halves * c_out), 30.0, F16)
    w = (w.float() * (torch.rand(w.shape, generator=g) < 1e-3)).to(F16)       # few: |z| stays small
    w[0] = 30.0
    x[:, 0] = normal(g, (n,), 2.0 ** -5, F16)
    dy = normal(g, (n, c_out), 2.0 ** -21, F16)
    dz, want = f16_gradients(halves, dy, x, w, None, "silu")
    back = smc.linear_backward if halves == 1 else smc.gated_backward
    got = back(dy.cuda(), x.cuda(), w.cuda(), activation="silu")
    for v, (wv, bd), label in zip(got, want, ("dx", "dw")):
        ro.check(v, wv, bd, label)


def test_f16_gradients_with_an_infinity():
    """One row of dy at infinity: its dx is not finite, every other row's is what
    it is without that row, also where dz is beyond f16."""
    g = gen(3)
    n, c_in, c_out = 300, 64, 72
    x, w = normal(g, (n, c_in), 0.1, F16), normal(g, (c_in, 2 * c_out), 2.0 ** -10, F16)
    b = torch.full((2 * c_out,), 300.0).to(F16)
    for size in (1.0, 500.0):
        dh = normal(g, (n, c_out), size, F16)
        clean = smc.gated_backward(dh.cuda(), x.cuda(), w.cuda(), bias=b.cuda())[0]
        assert torch.isfinite(clean).all()
        bad = dh.clone()
        bad[17, 5] = float("inf")
        dx = smc.gated_backward(bad.cuda(), x.cuda(), w.cuda(), bias=b.cuda())[0]
        keep = [i for i in range(n) if i != 17]
        assert not torch.isfinite(dx[17]).all()
        # (the largest finite value may be another one: a different power of two,
        # which the smallest values' rounding sees)
        top = clean.abs().max().item()
        assert (dx[keep].float() - clean[keep].float()).abs().max() <= 2.0 ** -10 * top


def test_f16_gradients_scale_in_a_graph():
    """The scale is found on the device: replays with small, ordinary and large
    gradients give the eager bits."""
    g = gen(4)
    n, c_in, c_out = 700, 64, 72
    x, w = normal(g, (n, c_in), 0.1, F16).cuda(), normal(g, (c_in, 2 * c_out), 2.0 ** -8, F16).cuda()
    b = torch.full((2 * c_out,), 300.0).to(F16).cuda()
    dh = torch.zeros(n, c_out, dtype=F16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        smc.gated_backward(dh, x, w, bias=b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = smc.gated_backward(dh, x, w, bias=b)
    for k, size in enumerate((1.0, 400.0, 2.0 ** -20, 0.1, 300.0)):
        fresh = normal(gen(50 + k), (n, c_out), size, F16).cuda()
        want = smc.gated_backward(fresh, x, w, bias=b)
        torch.cuda.synchronize()
        dh.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want)), size
        assert torch.isfinite(out[0]).all()


# ---- weight gradients over long row ranges --------------------------------------------
# Integers: every product and sum is exact in float32, so dw and db are equal bit
# for bit. The first four have as many ranges of the rows as the device takes (more
# than 256 rows each, the last one short); the last has more tiles than blocks.


@pytest.mark.parametrize("n,c_in,c_out,halves", [(91000, 128, 344, 2), (95000, 144, 256, 1), (131584, 128, 128, 1),
                                                 (15000, 512, 520, 2), (300, 3000, 3100, 1)])
def test_weight_gradient_ranges(n, c_in, c_out, halves):
    g = gen(n + c_in)
    x = torch.randint(-1, 2, (n, c_in), generator=g).to(BF16)
    dy = torch.randint(-1, 2, (n, c_out), generator=g).to(BF16)
    if halves == 1:
        w = torch.randint(-1, 2, (c_in, c_out), generator=g).to(BF16)
        b = torch.zeros(c_out, dtype=BF16)
        dz = dy.float()
        got = smc.linear_backward(dy.cuda(), x.cuda(), w.cuda(), bias=b.cuda())
    else:                                   # gate 2, up 1 for every row: dz = (dh, 2 dh)
        w = torch.zeros(c_in, 2 * c_out, dtype=BF16)
        b = torch.cat((torch.full((c_out,), 2.0), torch.full((c_out,), 1.0))).to(BF16)
        dz = torch.cat((dy.float(), 2 * dy.float()), 1)
        got = smc.gated_backward(dy.cuda(), x.cuda(), w.cuda(), bias=b.cuda(), activation="relu")
    assert torch.equal(got[0].cpu(), (dz @ w.float().t()).to(BF16))
    assert torch.equal(got[1].cpu(), (x.float().t() @ dz).to(BF16))
    assert torch.equal(got[2].cpu(), dz.sum(0).to(BF16))


# ---- rows of zeros without an epsilon ---------------------------------------------------


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,c", [(5, 7), (40, 128), (9, 512), (6, 1000), (4, 4104), (3, 4099)])
def test_norm_of_zero_rows_without_epsilon(n, c, dt):
    """eps = 0: a row of zeros stays zeros, in e4m3 with the smallest scale; its
    gradient is ds alone and it adds nothing to dweight. The other rows are as
    the formulas say."""
    g = gen(n * c)
    x, w, dy, ds = (normal(g, s, v, dt) for s, v in (((n, c), 1.0), ((c,), 1.0), ((n, c), 0.2), ((n, c), 0.5)))
    zero = torch.zeros(n, dtype=torch.bool)
    zero[::2] = True
    x[zero] = 0
    y, s = smc.rms_norm(x.cuda(), w.cuda(), residual=torch.zeros_like(x).cuda(), eps=0.0)
    assert torch.all(y[zero.cuda()] == 0) and torch.equal(s.cpu(), x)
    want, rel, _ = ro.norm(d(x[~zero]), None, d(w), 0.0)
    ro.check(y[(~zero).cuda()], want, ro.rounded(want, rel * want.abs(), dt), "y")
    q, scale = smc.rms_norm(x.cuda(), w.cuda(), eps=0.0, e4m3=True)
    q, scale = q.cpu().float(), scale.cpu()
    assert torch.all(q[zero] == 0) and torch.all(scale[zero] == 2.0 ** -126)
    assert torch.all(q[~zero].abs().amax(1) == 448)
    for extra in (None, ds):
        dx, dw = smc.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), eps=0.0, ds=None if extra is None else ds.cuda())
        at = zero.cuda()
        assert torch.equal(dx[at].cpu(), ds[zero]) if extra is not None else torch.all(dx[at] == 0)
        (wx, bx), (ww, bw) = ro.norm_backward(d(dy[~zero]), d(x[~zero]), d(w), 0.0,
                                              None if extra is None else d(ds[~zero]), dt)
        ro.check(dx[~at], wx, bx, "dx")
        ro.check(dw, ww, bw, "dweight")


# ---- more rows than one grid dimension counts threads --------------------------------


def room_for(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


@pytest.mark.parametrize("n,c,gib", [((1 << 26) + 131, 264, 40), ((1 << 24) + 3, 4104, 140)])
def test_norm_of_many_rows(n, c, gib):
    """Rows that take 2^32 threads and more, four rows a block and a block a row:
    every one is normalised, in place."""
    room_for(gib)
    x = torch.empty(n, c, dtype=BF16, device="cuda").fill_(3.0)
    w = torch.ones(c, dtype=BF16, device="cuda")
    assert norm_call(x, w, None, x, eps=0.0) == 0, smc.lib().smc_last_error()
    step = (1 << 30) // c
    for at in range(0, n, step):
        assert torch.all(x[at:at + step] == 1)
    del x
    torch.cuda.empty_cache()


def test_linear_of_many_unaligned_rows():
    """Rows of 1023 channels are copied to 1024 by more than 2^32 threads."""
    room_for(150)
    n, c, m = (1 << 25) + 77, 1023, 8
    x = torch.zeros(n, c, dtype=BF16, device="cuda")
    w = torch.zeros(c, m, dtype=BF16, device="cuda")
    w[c - 1] = torch.arange(1, m + 1)
    x[:, c - 1] = 1
    x[n - 1, c - 1] = 5
    x[1 << 24, 0] = 7
    w[0] = 1
    y = smc.linear(x, w)
    want = torch.arange(1, m + 1, device="cuda").to(BF16)
    assert torch.equal(y[n - 1], 5 * want) and torch.equal(y[1 << 24], want + 7)
    y[n - 1] = want
    y[1 << 24] = want
    assert torch.all(y == want)
    del x, y
    torch.cuda.empty_cache()


# ---- 8-bit weights ----------------------------------------------------------------------


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("c_in,c_out,extra", [(1, 1, 0), (7, 5, 0), (32, 32, 0), (33, 31, 3), (64, 200, 0),
                                              (513, 129, 8), (130, 1365, 1), (2048, 72, 0)])
def test_quantize_weight(c_in, c_out, extra, dt):
    """scale[j] = max(max |w[:, j]| / 448, 2^-126) and q[j, k] = e4m3(w[k, j] / scale[j])
    with float32 divisions and round to nearest even: the same bits as on the
    CPU. Columns of zeros, of the smallest values, with an infinity and with a NaN."""
    g = gen(c_in + c_out)
    wide = normal(g, (c_in, c_out + extra), 1.0, dt) * torch.logspace(-3, 2, c_out + extra).to(dt)
    w = wide[:, extra:]
    if c_out >= 31:
        w[:, 1] = 0
        w[:, 3] = 2.0 ** (-24 if dt == F16 else -130)
        w[0, 5], w[c_in - 1, 8] = float("inf"), float("nan")
    q, scale = smc.quantize_weight(wide.cuda()[:, extra:])
    assert q.shape == (c_out, c_in) and q.dtype == ro.E4M3 and scale.dtype == torch.float32
    f = w.float()
    want = (f.abs().amax(0) / 448).clamp(min=2.0 ** -126)
    if c_out >= 31:
        want[8] = float("nan")
    assert torch.equal(scale.cpu().nan_to_num(-1.0), want.nan_to_num(-1.0))
    ref, got = (f / want).t().to(ro.E4M3).float(), q.cpu().float()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got.nan_to_num(999.0), ref.nan_to_num(999.0))
    keep = torch.isfinite(want) & (f.abs().amax(0) >= 448 * 2.0 ** -126)
    assert torch.all(got[keep].abs().amax(1) == 448)


# ---- tiles ---------------------------------------------------------------------------------


@pytest.mark.parametrize("n,c_in,c_out", [(50000, 64, 72), (40000, 64, 72), (70000, 128, 40), (70000, 264, 104),
                                          (66000, 192, 264), (66000, 64, 520), (15000, 512, 384)])
def test_linear_in_every_tile(n, c_in, c_out):
    """Sizes on the sides of the rule that picks a tile; integers, bit for bit."""
    g = gen(n + c_in)
    x, w = (torch.randint(-1, 2, s, generator=g).to(BF16) for s in ((n, c_in), (c_in, c_out)))
    b, r = torch.randint(-3, 4, (c_out,), generator=g).to(BF16), torch.randint(-4, 5, (n, c_out), generator=g).to(BF16)
    z = (x.float() @ w.float() + b.float()).clamp(min=0)
    assert torch.equal(smc.linear(x.cuda(), w.cuda(), bias=b.cuda(), activation="relu").cpu(), z.to(BF16))
    y = smc.linear(x.cuda(), w.cuda(), bias=b.cuda(), residual=r.cuda(), activation="relu")
    assert torch.equal(y.cpu(), (z + r.float()).to(BF16))


@pytest.mark.parametrize("n", [2, 3, 4, 5, 7])
@pytest.mark.parametrize("c_in,c_out", [(64, 64), (768, 40), (776, 40), (1024, 72), (1032, 64), (2048, 200), (1030, 66)])
def test_few_rows_in_either_kernel(n, c_in, c_out):
    """Sizes on the sides of the rule that picks the few-row kernel."""
    for halves in (1, 2):
        g = gen(n + c_in + halves)
        x, w = normal(g, (n, c_in)), normal(g, (c_in, halves * c_out), c_in ** -0.5)
        b = normal(g, (halves * c_out,), 0.3)
        if halves == 1:
            r = normal(g, (n, c_out), 2.0)
            y = smc.linear(x.cuda(), w.cuda(), bias=b.cuda(), residual=r.cuda(), activation="silu")
            ro.check(y, *ro.linear(d(x), d(w), d(b), d(r), "silu", BF16), "linear")
        else:
            y = smc.gated(x.cuda(), w.cuda(), bias=b.cuda(), activation="silu")
            ro.check(y, *ro.gated(d(x), d(w), d(b), "silu", BF16), "gated")


def test_out_over_x_is_refused():
    x = normal(gen(1), (70, 64)).cuda()
    w = normal(gen(2), (64, 64), 0.1).cuda()
    want = smc.linear(x, w)
    for out in (x, x[:, :64]):
        with pytest.raises(smc.SmconvError):
            smc.linear(x, w, out=out)
    buf = torch.cat((x, x), 1)                  # columns of one buffer
    assert torch.equal(smc.linear(buf[:, :64], w, out=buf[:, 64:]), want)
    assert torch.equal(buf[:, :64], x)


@pytest.mark.parametrize("halves,size", [(1, 2.0 ** -22), (2, 2.0 ** -22), (1, 60000.0), (2, 3000.0)])
def test_f16_gradients_in_large_tiles(halves, size):
    """dz below and above f16's range in 128-row tiles of every product. Weights
    and x of powers of two, one nonzero weight a column and slopes of 1 (z far
    above 0): dz, dx and dw are sums of a few exact terms."""
    g = gen(halves)
    n, c, m = 15000, 512, 512
    x = torch.where(torch.rand(n, c, generator=g) < 0.5, -1.0, 1.0).to(F16) * 2.0 ** -10
    w = torch.zeros(c, halves * m, dtype=F16)
    w[torch.randint(0, c, (halves * m,), generator=g), torch.arange(halves * m)] = 2.0 ** -6
    b = torch.full((halves * m,), 1.0 if halves == 1 else 64.0).to(F16)
    dy = (torch.randint(-3, 4, (n, m), generator=g) * (size / 3)).to(F16)
    z = d(x) @ d(w) + d(b)
    dz = d(dy) if halves == 1 else torch.cat((d(dy) * z[:, m:], d(dy) * z[:, :m]), 1)
    assert z.min() > 0 and (dz.abs().max() > 65504 or dz.abs().max() < 2.0 ** -8 or halves == 1)
    back = smc.linear_backward if halves == 1 else smc.gated_backward
    dx, dw, _ = back(dy.cuda(), x.cuda(), w.cuda(), bias=b.cuda(), activation="relu")
    (wx, bx), (ww, bw), _ = ro.gradients(dz, dz.abs() * 2.0 ** -11 + dz.abs().max() * 2.0 ** -17, d(x), d(w), F16)
    for v, want, bound, label in ((dx, wx, bx, "dx"), (dw, ww, bw, "dw")):
        keep = want.abs() < 65000               # (a few sums are themselves beyond f16)
        assert keep.double().mean() > 0.99
        ro.check(v.cpu()[keep], want[keep], bound[keep], label)
