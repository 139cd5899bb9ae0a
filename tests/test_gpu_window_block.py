"""Group norm, projections and window attention together, as examples/window_block.py
runs them behind a convolution."""
import importlib.util
import math
import os

import pytest
import torch

import _rowops as ro

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location("window_block", os.path.join(ROOT, "examples", "window_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def formula(block, t, x, p, groups_of, windows_of, cells):
    """The block in float64 autograd."""
    n, c = t.shape
    y = torch.zeros_like(t)
    for rows in groups_of:
        v = t[rows].reshape(len(rows), block.GROUPS, -1)
        v = (v - v.mean((0, 2), keepdim=True)) / torch.sqrt(v.var((0, 2), unbiased=False, keepdim=True) + 1e-5)
        y = y.index_put((rows,), ro.act(v.reshape(len(rows), c) * p["norm"] + p["norm_bias"], "silu"))
    q, k, v = (y @ p["qkv"] + p["qkv_bias"]).chunk(3, 1)
    a = torch.zeros_like(t)
    h, largest, r = block.HEADS, 0.0, block.SIZE - 1
    for rows in windows_of:
        qw, kw, vw = (m[rows].view(len(rows), h, c // h).transpose(0, 1) for m in (q, k, v))
        s = (c // h) ** -0.5 * (qw @ kw.transpose(1, 2))
        apart = cells[rows][:, None] - cells[rows][None] + r
        for axis in range(3):
            s = s + p["table"][axis][apart[:, :, axis]].permute(2, 0, 1)
        largest = max(largest, s.detach().abs().max().item())
        a = a.index_put((rows,), (torch.softmax(s, 2) @ vw).transpose(0, 1).reshape(len(rows), c))
    return a @ p["out"] + p["out_bias"] + x, largest


@pytest.mark.parametrize("n,c,shift", [(1, 64, 0), (900, 64, 4), (700, 40, 0), (3000, 128, 0)])
def test_block_against_float64_autograd(block, n, c, shift):
    """Forward and every gradient of the whole block, by the norm of the difference. On its way out a value
    passes 5 roundings to bf16 (y, q k v, P, a, out), half an ulp (2^-8, relative) each, and q and k once more
    through the scores: 2^-8 of a score each, twice (numerator and sum), 4 |s| in all. On its way back a
    gradient passes 5 more (da, dS, dq dk dv, dy, dt or the weight's)."""
    g = torch.Generator()
    g.manual_seed(n + c)
    coords = block.make_cells(n, 2, (24, 16, 16), n)
    t, x = (torch.randn(n, c, generator=g).to(torch.bfloat16) for _ in range(2))
    dout = (torch.randn(n, c, generator=g) * 0.1).to(torch.bfloat16)
    w = block.make_weights(c, 3)
    for key in ("norm_bias", "qkv_bias", "out_bias", "table"):
        w[key] = (0.2 * torch.randn(w[key].shape, generator=g)).to(torch.bfloat16).cuda()
    windows, offsets = block.make_windows(coords, shift), block.sample_offsets(coords, 2)
    out, saved = block.forward(t.cuda(), x.cuda(), w, windows, offsets)
    dt, grads = block.backward(dout.cuda(), saved, w, windows, offsets)

    cells = coords.cpu().long()
    o = offsets.cpu().tolist()
    assert [int((cells[:, 0] < b).sum()) for b in range(3)] == o
    by = {}
    for i, row in enumerate(cells.tolist()):
        by.setdefault((row[0], *((v + shift) // block.SIZE for v in row[1:])), []).append(i)
    p = {k: v.cpu().double().requires_grad_(True) for k, v in w.items()}
    td, xd = t.double().requires_grad_(True), x.double().requires_grad_(True)
    samples = [torch.arange(a, b) for a, b in zip(o[:-1], o[1:]) if b > a]
    ref, largest = formula(block, td, xd, p, samples, [torch.tensor(v) for v in by.values()], cells[:, 1:])
    keys = list(p)
    want = torch.autograd.grad(ref, [td, xd] + [p[k] for k in keys], dout.double())
    ahead = (5 + 4 * largest) * 2.0 ** -8
    back = ahead + 5 * 2.0 ** -8

    def off(a, b):
        size = b.norm().item()
        return (a.double().cpu() - b).norm().item() / size if size else float(a.double().abs().max())

    assert off(out, ref.detach()) <= ahead
    assert off(dt, want[0]) <= back
    assert torch.equal(want[1], dout.double())
    for k, v in zip(keys, want[2:]):
        if n == 1 and k == "table":                 # a row alone: exactly none
            assert (grads[k] == 0).all() and (v.abs() < 1e-12).all()
        else:
            assert off(grads[k], v) <= back, k


def test_example_runs(block):
    losses = block.main(n=2000, steps=3)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
