"""Group norm at its edges: both sides of the one-launch rule, in place and captured, rows
far apart, as many samples as are taken, values of any size."""
import pytest
import torch

import _mixing as mx
import _rowops as ro
import submanifold_sparse_convolution_amd as smc
from test_gpu_group_norm import BF16, F16, device_offsets, inputs

pytestmark = pytest.mark.gpu


def run(x, w, b, dy, groups, o, name):
    y, stats = smc.group_norm(x, w, b, groups, offsets=o, activation=name, stats=True)
    return (y, stats, *smc.group_norm_backward(dy, x, w, b, groups, stats, offsets=o, activation=name))


# one launch up to 2,048 words of 8 channels
@pytest.mark.parametrize("n,c,groups,offsets", [(128, 128, 16, None), (129, 128, 16, None), (128, 128, 16, [3, 3, 80, 127]),
                                                (129, 128, 16, [0, 1, 129]), (2048, 8, 2, [0, 2000, 2048]), (2049, 1, 1, None),
                                                (2, 8192, 64, None), (3, 8192, 64, [0, 1, 3]), (2, 4104, 9, [1, 2])])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_one_launch_and_two(n, c, groups, offsets, dt):
    x, w, b, dy = inputs(n, c, dt, 7 * n + c)
    d = [t.double() for t in (x, w, b)]
    o = device_offsets(offsets)
    xc, wc, bc = x.cuda(), w.cuda(), b.cuda()
    y, stats, dx, dw, db = run(xc, wc, bc, dy.cuda(), groups, o, "silu")
    ro.check(y, *mx.group_norm(*d, groups, offsets, 1e-5, "silu", dt), "y")
    for got, (want, bound), label in zip((dx, dw, db), mx.group_norm_backward(dy.double(), *d, groups, stats.double().cpu(),
                                                                             offsets, "silu", dt), ("dx", "dw", "db")):
        ro.check(got, want, bound, label)
    # y over x, through the C entry
    a = smc.GroupNormArgs(n, c, groups, 1 if o is None else o.numel() - 1, 0 if dt == BF16 else 1, smc.ACTIVATIONS["silu"],
                          1e-5, None if o is None else o.data_ptr(), xc.data_ptr(), c, wc.data_ptr(), bc.data_ptr(),
                          xc.data_ptr(), c)
    a.workspace_bytes = smc.lib().smc_group_norm_workspace(a)
    ws = torch.empty(a.workspace_bytes, dtype=torch.uint8, device="cuda")
    a.workspace = ws.data_ptr()
    assert smc.lib().smc_group_norm(a, smc._raw_stream(xc.device)) == 0
    assert torch.equal(xc, y)


@pytest.mark.parametrize("n", [40, 1500])
def test_two_captured_calls(n):
    """Two calls in one graph, replayed on new rows and offsets between eager calls."""
    x, w, b, dy = (t.cuda() for t in inputs(n, 64, BF16, n))
    o = device_offsets([0, n // 3, n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one = run(x, w, b, dy, 8, o, "gelu")
        two = run(one[0], w, b, dy, 4, o, None)
    for k in range(4):
        fresh = inputs(n, 64, BF16, 60 + k)
        x.copy_(fresh[0])
        dy.copy_(fresh[3])
        o.copy_(torch.tensor([[0, n // 2, n], [0, 0, n], [5, 6, n - 1], [n, n, n]][k]))
        first = run(x, w, b, dy, 8, o, "gelu")
        second = run(first[0], w, b, dy, 4, o, None)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((*one, *two), (*first, *second)))


def test_rows_past_32_bit_offsets():
    """Rows 2^21 elements apart, 12 GB of them: the bits of rows side by side."""
    n, c = 3000, 64
    x, w, b, dy = (t.cuda() for t in inputs(n, c, BF16, 3))
    o = device_offsets([0, 1000, 3000])
    want = run(x, w, b, dy, 8, o, "silu")
    buf = torch.empty(n, 1 << 21, dtype=BF16, device="cuda")
    far, far_dy = buf[:, 64:128], buf[:, 1 << 20:(1 << 20) + 64]
    far.copy_(x)
    far_dy.copy_(dy)
    assert all(torch.equal(p, q) for p, q in zip(run(far, w, b, far_dy, 8, o, "silu"), want))


@pytest.mark.parametrize("rows", [1, 2])
def test_as_many_samples_as_are_taken(rows):
    """65,536 samples, a channel a group, equal rows in each: x_hat is 0, y the activation of the bias."""
    samples, c = 65536, 24
    _, w, b, _ = inputs(1, c, BF16, 4)
    x = torch.randn(samples, c, device="cuda").to(BF16).repeat_interleave(rows, 0)
    o = torch.arange(samples + 1, dtype=torch.int32, device="cuda") * rows
    y, stats = smc.group_norm(x, w.cuda(), b.cuda(), c, offsets=o, activation="silu", stats=True)
    want = ro.act(b.double(), "silu")
    ro.check(y[0], want, ro.rounded(want, ro.eval_err(b.double(), want), BF16), "y")
    assert torch.equal(y, y[:1].expand_as(y))
    assert torch.equal(stats[:, :, 0], x[::rows].float())
    dx, dw, db = smc.group_norm_backward(torch.ones_like(x), x, w.cuda(), b.cuda(), c, stats, offsets=o, activation="silu")
    assert (dw == 0).all() and (db != 0).all()
    if rows == 1:
        assert (dx == 0).all()
    with pytest.raises(smc.SmconvError, match="more than"):
        smc.group_norm(x, w.cuda(), b.cuda(), c, offsets=torch.zeros(65538, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("size,dt", [(2.0 ** -60, BF16), (2.0 ** 40, BF16), (2.0 ** 11, F16), (2.0 ** -12, F16)])
@pytest.mark.parametrize("n", [30, 700])
def test_values_of_any_size(size, dt, n):
    """Scaled by a power of two with eps scaled by its square (or none): the same y."""
    x, w, b, _ = inputs(n, 64, dt, 5)
    x = (x.float().clamp(-4, 4) * 0.5).to(dt)
    x = torch.where(x.abs() < 2.0 ** -2, torch.zeros_like(x), x)        # exact when scaled, in f16 too
    want = smc.group_norm(x.cuda(), w.cuda(), b.cuda(), 8, eps=0.0)
    got = smc.group_norm((x.double() * size).to(dt).cuda(), w.cuda(), b.cuda(), 8, eps=0.0)
    if size > 2.0 ** -50:
        assert torch.equal(got, want)
    else:                       # squares of 2^-60 stay normal float32 (2^-124 times a variance near 1)
        d = [t.double() for t in (x, w, b)]
        ro.check(got, *mx.group_norm(*d, 8, None, 0.0, None, dt), "y")
