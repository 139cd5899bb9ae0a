"""Window attention: values that are not finite in rows of no window and in masked keys,
probabilities below f16's normal numbers, scales at float32's lower end, rows without channels."""
import math

import pytest
import torch

import _mixing as mx
import _rowops as ro
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


@pytest.mark.parametrize("length,dim", [(30, 32), (64, 32), (100, 32), (500, 32), (30, 33), (100, 128)])
@pytest.mark.parametrize("cells", [False, True])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_a_key_that_is_masked_by_infinity(length, dim, cells, dt):
    """A key whose scores are all -inf in one head has no share there, as where they are merely far below the
    others: the same bits of out, dk (zeros for the key) and dv, also beside places that hold no query."""
    c = Case([length, 7], heads=4, kv=2, dim=dim, dt=dt, extent=(8, 8, 8) if cells else None, reach=3, order=False, seed=21)
    c.q[:, ::dim] = c.q[:, ::dim].abs() + 1
    c.k[5, 0] = -1e4
    q, k, v, table = (t if t is None else t.contiguous() for t in c.device())
    dout = c.dout.cuda()

    def run():
        out, lse = smc.window_attention(q, k, v, c.windows, 4, bias=table, lse=True)
        return (out, lse, *smc.window_attention_backward(dout, q, k, v, out, lse, c.windows, 4, bias=table))

    want = run()
    k[5, 0] = -math.inf
    got = run()
    for label, i in (("out", 0), ("lse", 1), ("dk", 3), ("dv", 4)):
        assert torch.equal(got[i], want[i]), label
    assert (got[3][5, :dim] == 0).all() and (got[4][5, :dim] == 0).all()
    if cells:
        assert torch.equal(got[5], want[5])


def test_f16_gradient_of_values_in_a_window_of_many_rows():
    """95,001 rows whose scores are alike: P is 1 / 95,001, below f16's normal numbers. With dout 1 every dv is 1.
    Half an ulp for P as an operand and one for dv, the additions of a step each, an exponential (2^-21), and lse, log 95,001."""
    n = 95001
    w = smc.Windows(torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    zero, one = (torch.full((n, 32), f, dtype=F16, device="cuda") for f in (0.0, 1.0))
    out, lse = smc.window_attention(zero, zero, one, w, 1, lse=True)
    _, _, dv, _ = smc.window_attention_backward(one, zero, zero, one, out, lse, w, 1)
    tol = 2 * 2.0 ** -11 + ro.gamma(n // 32 + 40) + 2.0 ** -21 + 4 * ro.U * math.log(n)
    assert ((dv.double() - 1).abs() <= tol).all()


def test_f16_gradient_of_values_with_little_weight():
    """Every query the same, keys' weights over a range of e^8 in a window of 20,000 rows: dv_j = n P_j, each to its own
    half ulps, down to P of 10^-8. Scores are exact products below 16 (their rounding and lse's: 4 u |s| each)."""
    n = 20000
    g = torch.Generator()
    g.manual_seed(22)
    w = smc.Windows(torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    q, k = torch.zeros(n, 32, dtype=F16), torch.zeros(n, 32, dtype=F16)
    q[:, 0] = 1
    k[:, 0] = (-8 * torch.rand(n, generator=g)).to(F16)
    v, one = (torch.full((n, 32), 1.0, dtype=F16, device="cuda") for _ in range(2))
    q, k = q.cuda(), k.cuda()
    out, lse = smc.window_attention(q, k, v, w, 1, scale=1.0, lse=True)
    _, _, dv, _ = smc.window_attention_backward(one, q, k, v, out, lse, w, 1, scale=1.0)
    want = n * torch.softmax(k[:, 0].double(), 0)
    tol = 2 * 2.0 ** -11 + ro.gamma(n // 32 + 40) + 2.0 ** -21 + 8 * ro.U * 16
    assert ((dv.double() - want[:, None]).abs() <= tol * want[:, None] + 2.0 ** -25).all()


@pytest.mark.parametrize("scale", [1e-45, 1e-40, 1e-38, 2.0 ** -100])
@pytest.mark.parametrize("cells", [False, True])
def test_scales_at_the_lower_end_of_float32(scale, cells):
    """Every score is the bias alone: out the mean of v under the softmax of the bias, lse with it."""
    c = Case([50, 130, 9], heads=4, kv=2, dim=32, extent=(8, 8, 8) if cells else None, reach=3, seed=23)
    q, k, v, table = c.device()
    args = list(c.formula())
    args[9] = 0.0
    want, bound, wl, el = mx.attention(*args)
    out, lse = smc.window_attention(q, k, v, c.windows, 4, bias=table, scale=scale, lse=True)
    ro.check(out, want, bound, "out")
    ro.check(lse, wl, el, "lse")


def test_rows_without_channels_are_refused():
    w = smc.Windows(torch.tensor([0, 4], dtype=torch.int32, device="cuda"), 4)
    none = torch.empty(4, 0, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="channels"):
        smc.window_attention(none, none, none, w, 2)


@pytest.mark.parametrize("first", [0, 50000, 95000])
def test_f16_output_of_many_keys_with_little_weight(first):
    """One key stands 12.16 above 95,000 others, whose weights of 5 10^-6 beside its own add up to half of it: out is their
    share. Half an ulp for P as an operand and one for out, the additions of a step each for the products and of four
    lanes for their sum, two exponentials (2^-21 each)."""
    n, top = 95001, 12.1640625
    w = smc.Windows(torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    q, k, v = (torch.zeros(n, 32, dtype=F16, device="cuda") for _ in range(3))
    q[:, 0], v[:] = 1, 1
    k[first, 0], v[first] = top, 0
    out = smc.window_attention(q, k, v, w, 1, scale=1.0)
    others = (n - 1) * math.exp(-top)
    tol = 2 * 2.0 ** -11 + ro.gamma(n // 32 + 80) + ro.gamma(n // 4 + 80) + 2 * 2.0 ** -21 + 8 * ro.U * top
    assert ((out.double() * (1 + others) / others - 1).abs() <= tol).all()


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("cells", [False, True])
def test_lse_of_many_keys_with_little_weight(dt, cells):
    """As above, the sum itself: weights are added up over a step (64 keys, 16 a lane), then to those before: n / 64 + 16
    additions after each other, and four lanes; half as many keys a step in short windows' blocks."""
    n, top = 95001, 12.0
    at = dict(coords=torch.zeros(n, 4, dtype=torch.int32, device="cuda"), extent=(1, 1, 1)) if cells else {}
    w = smc.Windows(torch.tensor([0, n], dtype=torch.int32, device="cuda"), n, **at)
    table = torch.zeros(3, 3, 1, dtype=dt, device="cuda") if cells else None
    q, k, v = (torch.zeros(n, 32, dtype=dt, device="cuda") for _ in range(3))
    q[:, 0], k[0, 0] = 1, top
    _, lse = smc.window_attention(q, k, v, w, 1, bias=table, scale=1.0, lse=True)
    others = (n - 1) * math.exp(-top)
    tol = ro.gamma(n // 32 + 80) + 2.0 ** -21 + 8 * ro.U * top
    assert ((lse.double() - top - math.log1p(others)).abs() <= tol).all()


@pytest.mark.parametrize("length", [30, 100, 700])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 12, 2.0 ** 15])
@pytest.mark.parametrize("cells", [False, True])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_scores_of_any_size(length, size, cells, dt):
    """Scores up to 2^35, whose neighbours in float32 are 2^12 apart: the largest takes all, wherever it stands among the
    keys, and the window's rows get its values to the bit."""
    g = torch.Generator()
    g.manual_seed(25)
    n = 4 * length
    at = dict(coords=torch.zeros(n, 4, dtype=torch.int32, device="cuda"), extent=(1, 1, 1)) if cells else {}
    w = smc.Windows(torch.arange(5, dtype=torch.int32, device="cuda") * length, n, **at)
    table = torch.full((3, 3, 2), 1.5, dtype=dt, device="cuda") if cells else None
    q = torch.full((n, 64), size, dtype=dt)
    k = torch.full((n, 64), size / 2, dtype=dt)
    top = torch.arange(4) * length + torch.tensor([0, length // 2, length - 1, 7])
    k[top] = size
    v = torch.randn(n, 64, generator=g).to(dt)
    out, lse = smc.window_attention(q.cuda(), k.cuda(), v.cuda(), w, 2, bias=table, scale=1.0, lse=True)
    assert torch.equal(out.cpu(), v[top].repeat_interleave(length, 0))
    want = 32 * size * size + (4.5 if cells else 0.0)
    assert ((lse.double() - want).abs() <= 4 * ro.U * want).all()


@pytest.mark.parametrize("first", [32768.0, 16384.0, 8192.0])
@pytest.mark.parametrize("length", [100, 700])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_a_key_little_above_large_scores(first, length, dt):
    """Scores of 2^25 (2^24, 2^23), scale log 2: a key of the window's last step stands 8 (powers of two) above one of its
    first, all others have no share. Exponents are exact but for the base's rounding, the same for both."""
    w = smc.Windows(torch.tensor([0, length], dtype=torch.int32, device="cuda"), length)
    q, k, v = (torch.zeros(length, 32, dtype=dt, device="cuda") for _ in range(3))
    q[:, 0], q[:, 1] = 1024, 8
    k[3, 0], k[3, 1], v[3] = first, 8, 1
    k[length - 2, 0], k[length - 2, 1], v[length - 2] = first, 9, 3
    out = smc.window_attention(q, k, v, w, 1, scale=math.log(2.0))
    want = (3 * 256 + 1) / 257
    tol = 2 * ro.HALF_ULP[dt] + ro.gamma(100) + 2 * 2.0 ** -21
    assert ((out.double() - want).abs() <= tol * want).all()


@pytest.mark.parametrize("first", [32768.0, 16384.0, 1024.0])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_gradients_beside_large_scores(first, dt):
    """One key above all others at scores of 2^25 (2^24, 2^20): P is 1 but for the rounding of its base, log2 e of the score,
    whose half ulp is 2 (1, 2^-5) powers of two, and as much again for lse. dv is that of the sum of dout, no infinity."""
    length = 100
    w = smc.Windows(torch.tensor([0, length], dtype=torch.int32, device="cuda"), length)
    q, k, v = (torch.zeros(length, 32, dtype=dt, device="cuda") for _ in range(3))
    q[:, 0] = 1024
    k[3, 0], v[3] = first, 1
    dout = torch.full_like(q, 2.0 ** -4)
    out, lse = smc.window_attention(q, k, v, w, 1, scale=1.0, lse=True)
    assert (out == 1).all()
    _, _, dv, _ = smc.window_attention_backward(dout, q, k, v, out, lse, w, 1, scale=1.0)
    off = (dv[3].double() / (length * 2.0 ** -4)).log2()
    assert (off.abs() <= {32768.0: 4, 16384.0: 2, 1024.0: 2.0 ** -4}[first] + 2 * ro.HALF_ULP[dt] * 1.5).all(), off
