"""Row operators (RMS norm, linear and gated layers) against their formulas in
64 bits: shapes that end inside tiles and words, single rows, strides,
alignments, streams, special values; integer-valued inputs bit for bit."""
import itertools

import pytest
import torch

import _rowops as ro
import submanifold_sparse_convolution_amd as smc

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
ACTS = (None, "relu", "silu", "gelu")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, shape, std=1.0, dt=BF16):
    return (torch.randn(shape, generator=g) * std).to(dt)


def ints(g, shape, lo, hi, dt=BF16):
    return torch.randint(lo, hi + 1, shape, generator=g).to(dt)


def d(t):
    return None if t is None else t.double()


def dev(t):
    return None if t is None else t.cuda()


def layer(seed, n, c_in, c_out, halves, dt, bias, std=1.0):
    g = gen(seed)
    x = normal(g, (n, c_in), std, dt)
    w = normal(g, (c_in, halves * c_out), c_in ** -0.5, dt)
    b = normal(g, (halves * c_out,), 0.3, dt) if bias else None
    return g, x, w, b


# rows x channels: single rows, odd sizes, both sides of every tile and word
SHAPES = [(1, 1, 1), (1, 512, 1365), (2, 8, 8), (3, 33, 17), (5, 200, 72), (16, 64, 64), (17, 65, 63),
          (31, 72, 200), (33, 128, 128), (64, 16, 344), (127, 520, 64), (129, 128, 129), (300, 344, 128),
          (513, 24, 40), (1000, 130, 250)]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,c_in,c_out", SHAPES)
def test_linear(n, c_in, c_out, dt):
    for k, (name, bias, residual) in enumerate(itertools.product(ACTS, (False, True), (False, True))):
        g, x, w, b = layer(17 * n + c_in + k, n, c_in, c_out, 1, dt, bias)
        r = normal(g, (n, c_out), 2.0, dt) if residual else None
        y = smc.linear(dev(x), dev(w), bias=dev(b), residual=dev(r), activation=name)
        assert y.dtype == dt
        want, bound = ro.linear(d(x), d(w), d(b), d(r), name, dt)
        ro.check(y, want, bound, f"{name} bias={bias} residual={residual}")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,c_in,c_out", SHAPES)
def test_gated(n, c_in, c_out, dt):
    for k, (name, bias) in enumerate(itertools.product(ACTS, (False, True))):
        g, x, w, b = layer(23 * n + c_in + k, n, c_in, c_out, 2, dt, bias)
        y = smc.gated(dev(x), dev(w), bias=dev(b), activation=name)
        want, bound = ro.gated(d(x), d(w), d(b), name, dt)
        ro.check(y, want, bound, f"{name} bias={bias}")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,c_in,c_out", SHAPES)
def test_linear_backward(n, c_in, c_out, dt):
    for k, (name, bias) in enumerate(itertools.product((None, "silu", "gelu"), (False, True))):
        g, x, w, b = layer(29 * n + c_in + k, n, c_in, c_out, 1, dt, bias)
        dy = normal(g, (n, c_out), 0.1, dt)
        got = smc.linear_backward(dev(dy), dev(x), dev(w), bias=dev(b), activation=name)
        assert (got[2] is None) == (b is None)
        want = ro.linear_backward(d(dy), d(x), d(w), d(b), name, dt)
        for v, (wv, bd), label in zip(got, want, ("dx", "dw", "db")):
            if v is not None:
                ro.check(v, wv, bd, f"{label} {name} bias={bias}")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,c_in,c_out", SHAPES)
def test_gated_backward(n, c_in, c_out, dt):
    for k, (name, bias) in enumerate(itertools.product((None, "silu", "gelu"), (False, True))):
        g, x, w, b = layer(31 * n + c_in + k, n, c_in, c_out, 2, dt, bias)
        dh = normal(g, (n, c_out), 0.1, dt)
        got = smc.gated_backward(dev(dh), dev(x), dev(w), bias=dev(b), activation=name)
        want = ro.gated_backward(d(dh), d(x), d(w), d(b), name, dt)
        for v, (wv, bd), label in zip(got, want, ("dx", "dw", "db")):
            if v is not None:
                ro.check(v, wv, bd, f"{label} {name} bias={bias}")


@pytest.mark.parametrize("n", [9, 12, 15, 16])
@pytest.mark.parametrize("c_in,c_out", [(64, 64), (65, 63), (2048, 40), (130, 1100)])
def test_few_rows(n, c_in, c_out):
    """More rows than one block of the few-row kernel takes."""
    g, x, w, b = layer(n + c_in, n, c_in, c_out, 1, BF16, True)
    r = normal(g, (n, c_out), 2.0)
    y = smc.linear(dev(x), dev(w), bias=dev(b), residual=dev(r), activation="silu")
    ro.check(y, *ro.linear(d(x), d(w), d(b), d(r), "silu", BF16), "linear")
    g, x, w, b = layer(n + c_in, n, c_in, c_out, 2, BF16, True)
    y = smc.gated(dev(x), dev(w), bias=dev(b), activation="gelu")
    ro.check(y, *ro.gated(d(x), d(w), d(b), "gelu", BF16), "gated")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,c_in,c_out", [(17, 65, 63), (40, 64, 50), (300, 33, 56), (2500, 141, 141), (4200, 72, 525)])
def test_unaligned_rows_without_workspace(n, c_in, c_out, dt):
    """The C entries read rows that are not whole 16-byte words in place where
    they are given no room for copies; both forms agree with the formulas."""
    L = smc.lib()
    for halves, entry, need in ((1, L.smc_linear, L.smc_linear_workspace), (2, L.smc_gated, L.smc_gated_workspace)):
        g, x, w, b = layer(n + c_in, n, c_in, c_out, halves, dt, True)
        xd, wd, bd = dev(x), dev(w), dev(b)
        want = (ro.linear(d(x), d(w), d(b), None, "silu", dt) if halves == 1 else
                ro.gated(d(x), d(w), d(b), "silu", dt))
        a, _, shape = smc._product_args(halves, xd, wd, bd, "silu", None, None, None)
        y = smc._product_out(a, xd, None, dt, shape)
        nbytes = need(a)
        assert nbytes > 0 or c_in <= 64         # no copies for a single step
        for ws in (None, torch.full((max(nbytes, 16),), 255, dtype=torch.uint8, device="cuda")):
            y.fill_(float("nan"))
            if ws is not None:
                a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes
            assert entry(a, smc._raw_stream(xd.device)) == 0
            ro.check(y, *want, f"halves={halves} workspace={ws is not None}")


# Sizes of every tile shape, tails of rows, columns and contraction. Integers:
# every product and sum is exact in float32, so the one rounding left is the
# output's (and dz's), and results are equal bit for bit.
EXACT = [(1, 40, 24), (7, 64, 72), (64, 128, 256), (130, 72, 130), (700, 200, 96), (2500, 96, 344),
         (9000, 64, 264), (33000, 128, 128), (3000, 512, 520)]


@pytest.mark.parametrize("n,c_in,c_out", EXACT)
def test_linear_exact(n, c_in, c_out):
    g = gen(n + c_in)
    x, w = ints(g, (n, c_in), -2, 2), ints(g, (c_in, c_out), -1, 1)
    b, r = ints(g, (c_out,), -3, 3), ints(g, (n, c_out), -4, 4)
    z = x.float() @ w.float() + b.float()
    y = smc.linear(dev(x), dev(w), bias=dev(b), residual=dev(r), activation="relu")
    assert torch.equal(y.cpu(), (z.clamp(min=0) + r.float()).to(BF16))
    # backward with the slopes exact too: dz = dy or 0
    dy = ints(g, (n, c_out), -1, 1)
    dz = dy.float() * (z > 0)
    got = smc.linear_backward(dev(dy), dev(x), dev(w), bias=dev(b), activation="relu")
    assert torch.equal(got[0].cpu(), (dz @ w.float().t()).to(BF16))
    assert torch.equal(got[1].cpu(), (x.float().t() @ dz).to(BF16))
    assert torch.equal(got[2].cpu(), dz.sum(0).to(BF16))


@pytest.mark.parametrize("n,c_in,c_out", EXACT)
def test_gated_exact(n, c_in, c_out):
    g = gen(n + c_in + 1)
    x, w = ints(g, (n, c_in), -1, 1), ints(g, (c_in, 2 * c_out), -1, 1)
    b = ints(g, (2 * c_out,), -3, 3)
    z = x.float() @ w.float() + b.float()
    gate, up = z[:, :c_out], z[:, c_out:]
    h = smc.gated(dev(x), dev(w), bias=dev(b), activation="relu")
    assert torch.equal(h.cpu(), (gate.clamp(min=0) * up).to(BF16))
    dh = ints(g, (n, c_out), -1, 1)
    dz = torch.cat((dh.float() * up * (gate > 0), dh.float() * gate.clamp(min=0)), 1).to(BF16).double()
    got = smc.gated_backward(dev(dh), dev(x), dev(w), bias=dev(b), activation="relu")
    # |dz| <= 515 and at most 33,000 terms: sums below 2^24, exact
    assert torch.equal(got[0].cpu(), (dz @ w.double().t()).float().to(BF16))
    assert torch.equal(got[1].cpu(), (x.double().t() @ dz).float().to(BF16))
    assert torch.equal(got[2].cpu(), dz.sum(0).float().to(BF16))


@pytest.mark.parametrize("transposed", [True, False])
@pytest.mark.parametrize("n,c_in,c_out", [(1, 512, 40), (3, 33, 17), (65, 16, 169), (300, 128, 128),
                                          (130, 200, 72), (5000, 256, 344), (129, 1040, 130)])
def test_e4m3_layers(n, c_in, c_out, transposed):
    """e4m3 operands are exact inputs: the bound is the 16-bit layers' with the
    scales' products and the e4m3 instruction's own loss added."""
    for halves, dt, name in ((1, BF16, "gelu"), (2, BF16, "silu"), (1, F16, None), (2, F16, "gelu")):
        g = gen(n + c_in + halves)
        q, xs = smc.rms_norm(dev(normal(g, (n, c_in))), torch.ones(c_in, dtype=BF16, device="cuda"), e4m3=True)
        w = dev(normal(g, (c_in, halves * c_out), c_in ** -0.5))
        wq, ws = smc.quantize_weight(w)
        assert wq.shape == (halves * c_out, c_in)
        if not transposed:
            wq = wq.t().contiguous().t()
        b = normal(g, (halves * c_out,), 0.3, dt)
        xd = q.cpu().double() * xs.cpu().double()[:, None]
        wd = (wq.cpu().double() * ws.cpu().double()[:, None]).t()
        if halves == 1:
            r = normal(g, (n, c_out), 1.0, dt)
            y = smc.linear(q, wq, bias=dev(b), residual=dev(r), activation=name, x_scale=xs, w_scale=ws, dtype=dt)
            z, ez = ro.pre(xd, wd, d(b), extra_terms=5, loss=ro.E4M3_LOSS)
            v = ro.act(z, name)
            want = v + d(r)
            err = 1.13 * ez + ro.eval_err(z, v) + ro.U * want.abs()
        else:
            y = smc.gated(q, wq, bias=dev(b), activation=name, x_scale=xs, w_scale=ws, dtype=dt)
            z, ez = ro.pre(xd, wd, d(b), extra_terms=5, loss=ro.E4M3_LOSS)
            gt, up, eg, eu = z[:, :c_out], z[:, c_out:], ez[:, :c_out], ez[:, c_out:]
            a = ro.act(gt, name)
            ea = 1.13 * eg + ro.eval_err(gt, a)
            want = a * up
            err = ea * up.abs() + a.abs() * eu + ea * eu + 2 * ro.U * want.abs()
        assert y.dtype == dt
        ro.check(y, want, ro.rounded(want, err, dt), f"halves={halves} {name}")


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("n,c_in,c_out", [(1, 145, 33), (20, 1488, 106), (40, 130, 50), (300, 530, 300), (2500, 241, 141)])
def test_unaligned_e4m3_without_workspace(n, c_in, c_out, transposed):
    """e4m3 rows that are not whole 16-byte words, in place and through copies,
    w in both memory orders."""
    L = smc.lib()
    for halves, entry, need in ((1, L.smc_linear, L.smc_linear_workspace), (2, L.smc_gated, L.smc_gated_workspace)):
        g = gen(n + c_in + halves)
        q, xs = smc.rms_norm(dev(normal(g, (n, c_in))), torch.ones(c_in, dtype=BF16, device="cuda"), e4m3=True)
        wq, ws = smc.quantize_weight(dev(normal(g, (c_in, halves * c_out), c_in ** -0.5)))
        if not transposed:
            wq = wq.t().contiguous().t()
        b = normal(g, (halves * c_out,), 0.3)
        xd = q.cpu().double() * xs.cpu().double()[:, None]
        wd = (wq.cpu().double() * ws.cpu().double()[:, None]).t()
        z, ez = ro.pre(xd, wd, d(b), extra_terms=5, loss=ro.E4M3_LOSS)
        if halves == 1:
            want, err = z, ez
        else:
            a = ro.act(z[:, :c_out], "relu")
            want = a * z[:, c_out:]
            err = ez[:, :c_out] * z[:, c_out:].abs() + a * ez[:, c_out:] + ez[:, :c_out] * ez[:, c_out:] + ro.U * want.abs()
        bound = ro.rounded(want, err, BF16)
        args, dt, shape = smc._product_args(halves, q, wq, dev(b), None if halves == 1 else "relu", xs, ws, BF16)
        bias = dev(b)
        args.bias = bias.data_ptr()
        y = smc._product_out(args, q, None, dt, shape)
        nbytes = need(args)
        for room in (None, torch.full((max(nbytes, 16),), 255, dtype=torch.uint8, device="cuda")):
            y.fill_(float("nan"))
            if room is not None:
                args.workspace, args.workspace_bytes = room.data_ptr(), nbytes
            assert entry(args, smc._raw_stream(q.device)) == 0
            ro.check(y, want, bound, f"halves={halves} workspace={room is not None} ({nbytes} bytes)")


def test_e4m3_exact():
    """Small integers are e4m3 values; powers of two as scales: bit for bit."""
    g = gen(5)
    n, c_in, c_out = 700, 144, 200
    x, w = ints(g, (n, c_in), -3, 3), ints(g, (c_out, c_in), -2, 2)
    xs = torch.tensor([1.0, 0.5, 4.0])[torch.randint(0, 3, (n,), generator=g)]
    ws = torch.tensor([2.0, 0.25])[torch.randint(0, 2, (c_out,), generator=g)]
    want = ((x.float() * xs[:, None]) @ (w.float() * ws[:, None]).t()).to(BF16)
    for wq in (w.to(ro.E4M3).cuda(), w.t().contiguous().to(ro.E4M3).cuda().t()):
        y = smc.linear(x.to(ro.E4M3).cuda(), wq, x_scale=xs.cuda(), w_scale=ws.cuda())
        assert torch.equal(y.cpu(), want)


# ---- norm ----------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (1, 512), (2, 7), (3, 8), (5, 16), (63, 33), (64, 64), (65, 72), (100, 128), (33, 130),
               (40, 200), (17, 256), (12, 344), (9, 512), (7, 520), (6, 1000), (5, 1024), (4, 1025), (3, 2048),
               (5, 2056), (2, 4096), (3, 4104), (2, 8200), (2, 4099), (1000, 128), (4500, 16)]


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,c", NORM_SHAPES)
def test_rms_norm(n, c, dt):
    g = gen(n + c)
    x, r, w = normal(g, (n, c), 1.0, dt), normal(g, (n, c), 2.0, dt), normal(g, (c,), 1.0, dt)
    for res in (None, r):
        got = smc.rms_norm(dev(x), dev(w), residual=dev(res), eps=1e-5)
        y = got if res is None else got[0]
        want, rel, s = ro.norm(d(x), d(res), d(w), 1e-5)
        ro.check(y, want, ro.rounded(want, rel * want.abs(), dt), "y")
        if res is not None:
            ro.check(got[1], s, ro.rounded(s, ro.U * s.abs(), dt), "s")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,c", NORM_SHAPES)
def test_rms_norm_e4m3(n, c, dt):
    g = gen(n + c + 7)
    x, r, w = normal(g, (n, c), 1.0, dt), normal(g, (n, c), 2.0, dt), normal(g, (c,), 1.0, dt)
    for res in (None, r):
        q, scale, *s_out = smc.rms_norm(dev(x), dev(w), residual=dev(res), e4m3=True)
        assert q.dtype == ro.E4M3 and scale.dtype == torch.float32 and len(s_out) == (res is not None)
        want, rel, s = ro.norm(d(x), d(res), d(w), 1e-6)
        ws = (want.abs().amax(1) / 448).clamp(min=2.0 ** -126)
        ro.check(scale, ws, (rel + 2 * ro.U) * ws, "scale")
        # half an e4m3 ulp of the scaled value: 2^-4 relative, 2^-10 below 2^-6
        v = want / ws[:, None]
        slack = (2 * rel + 4 * ro.U) * v.abs()
        ro.check(q.float(), v, slack + torch.maximum(2.0 ** -4 * (v.abs() + slack), torch.tensor(2.0 ** -10).double()),
                 "q")
        assert torch.all(q.float().abs().amax(1) == 448)
        if res is not None:
            ro.check(s_out[0], s, ro.rounded(s, ro.U * s.abs(), dt), "s")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("n,c", NORM_SHAPES + [(20000, 64)])
def test_rms_norm_backward(n, c, dt):
    g = gen(n + c + 9)
    s, dy, w = normal(g, (n, c), 1.5, dt), normal(g, (n, c), 0.2, dt), normal(g, (c,), 1.0, dt)
    ds = normal(g, (n, c), 0.5, dt)
    for extra in (None, ds):
        dx, dw = smc.rms_norm_backward(dev(dy), dev(s), dev(w), eps=1e-5, ds=dev(extra))
        (wx, bx), (ww, bw) = ro.norm_backward(d(dy), d(s), d(w), 1e-5, d(extra), dt)
        ro.check(dx, wx, bx, "dx")
        ro.check(dw, ww, bw, "dweight")


def test_norm_of_zeros_and_special_rows():
    x = torch.zeros(4, 128, dtype=BF16)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 1.0
    w = torch.ones(128, dtype=BF16)
    y = smc.rms_norm(x.cuda(), w.cuda(), eps=0.0 + 1e-6).cpu().float()
    assert torch.all(y[0] == 0)
    assert torch.all(torch.isnan(y[1]))
    assert torch.isnan(y[2, 7]) and torch.all(torch.cat((y[2, :7], y[2, 8:])) == 0)
    assert torch.all(y[3] == 1)
    q, scale = smc.rms_norm(x.cuda(), w.cuda(), e4m3=True)
    q, scale = q.cpu().float(), scale.cpu()
    assert torch.all(q[0] == 0) and scale[0] == 2.0 ** -126
    assert torch.isnan(scale[1]) and torch.all(torch.isnan(q[1]))
    assert torch.isnan(scale[2])
    assert torch.all(q[3] == 448)


def test_special_values_stay_in_their_rows():
    """An infinity or NaN in one row of x reaches that row of y alone, also
    where tiles are padded; relu keeps NaN."""
    g, x, w, b = layer(3, 70, 72, 40, 1, BF16, True)
    clean = smc.linear(dev(x), dev(w), bias=dev(b), activation="relu")
    x2 = x.clone()
    x2[69] = float("nan")
    x2[10, 71] = float("inf")
    y = smc.linear(dev(x2), dev(w), bias=dev(b), activation="relu")
    assert torch.all(torch.isnan(y[69]))
    keep = [i for i in range(70) if i not in (10, 69)]
    assert torch.equal(y[keep], clean[keep])
    z = (x2[10].float() @ w.float())
    want = torch.where(z < 0, torch.zeros_like(z), z)
    assert torch.equal(torch.isinf(y[10].cpu().float()), torch.isinf(want))


# ---- strides, alignment, streams ---------------------------------------------------


def strided(t, left, right, skip=2):
    """t as a view: columns left .. of wider rows, every `skip`-th row; what lies
    between holds NaN."""
    n, c = t.shape
    if t.dtype == ro.E4M3:
        wide = torch.full((n * skip, left + c + right), 0x7f, dtype=torch.uint8).view(ro.E4M3).cuda()
    else:
        wide = torch.full((n * skip, left + c + right), float("nan"), dtype=t.dtype, device="cuda")
    v = wide[::skip, left:left + c]
    v.copy_(t.cuda())
    return v


@pytest.mark.parametrize("left,right", [(0, 0), (8, 8), (16, 3), (1, 0), (3, 5)])
@pytest.mark.parametrize("n,c_in,c_out", [(1, 64, 40), (9, 72, 64), (70, 64, 136), (40, 33, 50), (600, 128, 64)])
def test_views(n, c_in, c_out, left, right):
    """Views give what contiguous copies give, bit for bit where the same kernel
    runs, else within the bound; the NaN around them is not touched."""
    for halves in (1, 2):
        g, x, w, b = layer(n + left, n, c_in, c_out, halves, BF16, True)
        r, dy = normal(g, (n, c_out)), normal(g, (n, c_out), 0.1)
        xv, wv, rv, dyv = (strided(t, left, right) for t in (x, w, r, dy))
        out = strided(torch.zeros(n, c_out, dtype=BF16), left, right)
        base = out._base if out._base is not None else out
        mask = torch.ones_like(base, dtype=torch.bool)
        mask[::2, left:left + c_out] = False
        if halves == 1:
            got = smc.linear(xv, wv, bias=dev(b), residual=rv, activation="silu", out=out)
            want, bound = ro.linear(d(x), d(w), d(b), d(r), "silu", BF16)
            back = smc.linear_backward(dyv, xv, wv, bias=dev(b), activation="silu")
            wb = ro.linear_backward(d(dy), d(x), d(w), d(b), "silu", BF16)
        else:
            got = smc.gated(xv, wv, bias=dev(b), activation="silu", out=out)
            want, bound = ro.gated(d(x), d(w), d(b), "silu", BF16)
            back = smc.gated_backward(dyv, xv, wv, bias=dev(b), activation="silu")
            wb = ro.gated_backward(d(dy), d(x), d(w), d(b), "silu", BF16)
        assert got is out
        ro.check(out, want, bound, f"y halves={halves}")
        if n > 1:
            assert torch.all(torch.isnan(base[mask]))
        for v, (wvv, bd), label in zip(back, wb, ("dx", "dw", "db")):
            ro.check(v, wvv, bd, f"{label} halves={halves}")


@pytest.mark.parametrize("left,right", [(0, 0), (8, 8), (1, 0), (3, 5)])
@pytest.mark.parametrize("n,c", [(1, 64), (9, 72), (70, 128), (40, 33), (5, 4104)])
def test_norm_views(n, c, left, right):
    g = gen(n + c)
    x, r, dy, w = normal(g, (n, c)), normal(g, (n, c)), normal(g, (n, c), 0.1), normal(g, (c,))
    xv, rv, dyv = (strided(t, left, right) for t in (x, r, dy))
    y, s = smc.rms_norm(xv, dev(w), residual=rv)
    want, rel, sw = ro.norm(d(x), d(r), d(w), 1e-6)
    ro.check(y, want, ro.rounded(want, rel * want.abs(), BF16), "y")
    ro.check(s, sw, ro.rounded(sw, ro.U * sw.abs(), BF16), "s")
    dx, dw = smc.rms_norm_backward(dyv, xv, dev(w), ds=rv)
    (wx, bx), (ww, bw) = ro.norm_backward(d(dy), d(x), d(w), 1e-6, d(r), BF16)
    ro.check(dx, wx, bx, "dx")
    ro.check(dw, ww, bw, "dweight")


@pytest.mark.parametrize("left,right", [(0, 0), (16, 16), (1, 0), (8, 8)])
def test_e4m3_views(left, right):
    g = gen(77)
    n, c_in, c_out = 70, 80, 48
    x, w = ints(g, (n, c_in), -3, 3), ints(g, (c_out, c_in), -2, 2)
    ones = torch.ones(n, device="cuda"), torch.ones(c_out, device="cuda")
    want = (x.float() @ w.float().t()).to(BF16)
    xv, wv = strided(x.to(ro.E4M3), left, right), strided(w.to(ro.E4M3), left, right)
    wt = strided(w.t().contiguous().to(ro.E4M3), left, right).t()
    for ww in (wv, wt):
        assert torch.equal(smc.linear(xv, ww, x_scale=ones[0], w_scale=ones[1]).cpu(), want)


def test_out_is_the_residual():
    g, x, w, b = layer(1, 300, 128, 96, 1, BF16, True)
    r = normal(g, (300, 96))
    want = smc.linear(dev(x), dev(w), bias=dev(b), residual=dev(r), activation="gelu")
    buf = dev(r)
    assert smc.linear(dev(x), dev(w), bias=dev(b), residual=buf, activation="gelu", out=buf) is buf
    assert torch.equal(buf, want)


def test_empty_rows():
    w = torch.randn(64, 32, device="cuda").to(BF16)
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    assert smc.linear(x, w).shape == (0, 32)
    assert smc.gated(x, w).shape == (0, 16)
    dx, dw, db = smc.linear_backward(torch.empty(0, 32, dtype=BF16, device="cuda"), x, w,
                                     bias=torch.zeros(32, dtype=BF16, device="cuda"), activation="silu")
    assert dx.shape == (0, 64) and torch.all(dw == 0) and torch.all(db == 0) and dw.shape == (64, 32)
    dx, dw, db = smc.gated_backward(torch.empty(0, 16, dtype=BF16, device="cuda"), x, w)
    assert dx.shape == (0, 64) and torch.all(dw == 0) and db is None
    wn = torch.ones(64, dtype=BF16, device="cuda")
    y, s = smc.rms_norm(x, wn, residual=x)
    assert y.shape == s.shape == (0, 64)
    q, scale = smc.rms_norm(x, wn, e4m3=True)
    assert q.shape == (0, 64) and scale.shape == (0,)
    dx, dwn = smc.rms_norm_backward(x, x, wn)
    assert dx.shape == (0, 64) and torch.all(dwn == 0)


def test_other_stream():
    """A call on a given stream reads inputs and writes outputs in that
    stream's order (waited for by events, no device synchronisation)."""
    g, x, w, b = layer(2, 4000, 128, 128, 2, BF16, True)
    x, w, b = dev(x), dev(w), dev(b)
    dh = dev(normal(g, (4000, 128), 0.1))
    want = (smc.gated(x, w, bias=b),) + smc.gated_backward(dh, x, w, bias=b)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = (smc.gated(x, w, bias=b, stream=st),) + smc.gated_backward(dh, x, w, bias=b, stream=st)
        torch.cuda.current_stream().wait_stream(st)
        for a, c in zip(got, want):
            assert torch.equal(a, c)


def test_equal_inputs_give_equal_bits():
    g, x, w, b = layer(4, 30000, 128, 128, 2, BF16, True)
    x, w, b = dev(x), dev(w), dev(b)
    dh = dev(normal(g, (30000, 128), 0.1))
    wn = torch.ones(128, dtype=BF16, device="cuda")
    first = smc.gated_backward(dh, x, w, bias=b) + smc.rms_norm_backward(dh, x, wn)
    for _ in range(5):
        again = smc.gated_backward(dh, x, w, bias=b) + smc.rms_norm_backward(dh, x, wn)
        assert all(torch.equal(a, c) for a, c in zip(first, again))


def test_graph_replays():
    """Forward and backward captured in a HIP graph: every replay, with new
    input values and eager work in between, equals the eager result."""
    g, x, w, b = layer(6, 3000, 128, 96, 2, BF16, True)
    x, w, b = dev(x), dev(w), dev(b)
    wn = torch.ones(128, dtype=BF16, device="cuda")
    w2 = dev(normal(g, (96, 128), 0.1))

    def step(x):
        y, s = smc.rms_norm(x, wn, residual=x)
        h = smc.gated(y, w, bias=b)
        o = smc.linear(h, w2, residual=s)
        dh, dw2, _ = smc.linear_backward(o, h, w2)
        return (o, dw2) + smc.gated_backward(dh, y, w, bias=b)

    xs = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(xs)
    for k in range(4):
        xn = dev(normal(gen(100 + k), (3000, 128)))
        want = step(xn)
        torch.cuda.synchronize()
        xs.copy_(xn)
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, want):
            assert torch.equal(a, c)


# ---- gradients against differences ---------------------------------------------------


def test_gradients_match_differences():
    """dL of L = sum(dy y) along random directions, from the float64 formulas of
    the forward pass, against the kernels' gradients. Central differences of a
    smooth function with step 1e-4 are exact to 1e-7 here; the gradients carry
    the roundings of dz and of the outputs, random in sign: within
    4 sqrt(sum of squared rounding bounds) of the sum."""
    g, x, w, b = layer(8, 50, 48, 40, 2, F16, True)
    dh = normal(g, (50, 40), 0.5, F16)
    got = smc.gated_backward(dev(dh), dev(x), dev(w), bias=dev(b), activation="gelu")
    bounds = [bd for _, bd in ro.gated_backward(d(dh), d(x), d(w), d(b), "gelu", F16)]
    ops = [d(x), d(w), d(b)]

    def loss(x, w, b):
        z = x @ w + b
        return (d(dh) * ro.act(z[:, :40], "gelu") * z[:, 40:]).sum()

    for i, grad in enumerate(got):
        v = torch.randn(ops[i].shape, generator=g, dtype=torch.float64)
        lo, hi = list(ops), list(ops)
        hi[i], lo[i] = ops[i] + 1e-4 * v, ops[i] - 1e-4 * v
        want = (loss(*hi) - loss(*lo)) / 2e-4
        have = (grad.double().cpu() * v).sum()
        tol = 4 * ((bounds[i] * v) ** 2).sum().sqrt() + 1e-5 * want.abs() + 1e-5
        assert (have - want).abs() <= tol, (i, have.item(), want.item(), tol.item())


def test_norm_gradients_match_differences():
    g = gen(12)
    s, dy, w = normal(g, (40, 72), 1.0, F16), normal(g, (40, 72), 0.5, F16), normal(g, (72,), 1.0, F16)
    got = smc.rms_norm_backward(dev(dy), dev(s), dev(w), eps=1e-3)
    bounds = [bd for _, bd in ro.norm_backward(d(dy), d(s), d(w), 1e-3, None, F16)]
    ops = [d(s), d(w)]

    def loss(s, w):
        return (d(dy) * ro.norm(s, None, w, 1e-3)[0]).sum()

    for i, grad in enumerate(got):
        v = torch.randn(ops[i].shape, generator=g, dtype=torch.float64)
        lo, hi = list(ops), list(ops)
        hi[i], lo[i] = ops[i] + 1e-4 * v, ops[i] - 1e-4 * v
        want = (loss(*hi) - loss(*lo)) / 2e-4
        have = (grad.double().cpu() * v).sum()
        tol = 4 * ((bounds[i] * v) ** 2).sum().sqrt() + 1e-5 * want.abs() + 1e-5
        assert (have - want).abs() <= tol, (i, have.item(), want.item(), tol.item())


# ---- refusals -----------------------------------------------------------------------


def test_refusals():
    x = torch.zeros(4, 16, dtype=BF16, device="cuda")
    w = torch.zeros(16, 8, dtype=BF16, device="cuda")
    wn = torch.zeros(16, dtype=BF16, device="cuda")
    bad = [
        (TypeError, lambda: smc.linear(x.cpu(), w)),
        (TypeError, lambda: smc.linear(x.float(), w)),
        (TypeError, lambda: smc.linear(x, w.half())),
        (ValueError, lambda: smc.linear(x[0], w)),
        (ValueError, lambda: smc.linear(x, w[:8])),
        (ValueError, lambda: smc.linear(x.t().contiguous().t(), w)),
        (ValueError, lambda: smc.linear(x[:1].expand(4, 16), w)),
        (ValueError, lambda: smc.linear(x, w, bias=wn)),
        (TypeError, lambda: smc.linear(x, w, bias=wn[:8].float())),
        (ValueError, lambda: smc.linear(x, w, residual=x)),
        (ValueError, lambda: smc.linear(x, w, activation="tanh")),
        (ValueError, lambda: smc.linear(x, w, x_scale=torch.ones(4, device="cuda"))),
        (ValueError, lambda: smc.linear(x, w, dtype=F16)),
        (ValueError, lambda: smc.linear(x, w, out=x)),
        (ValueError, lambda: smc.gated(x, w[:, :7])),
        (ValueError, lambda: smc.linear_backward(x, x, w)),
        (ValueError, lambda: smc.rms_norm(x, wn[:8])),
        (ValueError, lambda: smc.rms_norm(x, wn, residual=x[:3])),
        (TypeError, lambda: smc.rms_norm(x, wn, residual=x.half())),
        (smc.SmconvError, lambda: smc.rms_norm(x, wn, eps=-1.0)),
        (smc.SmconvError, lambda: smc.rms_norm(x, wn, eps=float("nan"))),
        (ValueError, lambda: smc.rms_norm_backward(x[:2], x, wn)),
        (TypeError, lambda: smc.linear(x.to(ro.E4M3), w.t().contiguous().to(ro.E4M3))),       # no scales
        (TypeError, lambda: smc.linear(x.to(ro.E4M3), w, x_scale=torch.ones(4, device="cuda"),
                                       w_scale=torch.ones(8, device="cuda"))),
        (smc.SmconvError, lambda: smc.linear_backward(
            torch.zeros(4, 8, dtype=BF16, device="cuda"), x.to(ro.E4M3), w.t().contiguous().to(ro.E4M3))),
        (TypeError, lambda: smc.quantize_weight(w.float())),
    ]
    for k, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"case {k} was accepted")
