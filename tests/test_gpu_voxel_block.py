"""The row operators together, as examples/voxel_block.py runs them."""
import importlib.util
import os

import pytest
import torch

import _rowops as ro

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location("voxel_block", os.path.join(ROOT, "examples", "voxel_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("n,c,hidden", [(1, 64, 176), (777, 64, 176), (3000, 128, 344), (500, 33, 50)])
def test_block_against_float64_autograd(block, n, c, hidden):
    """Forward and every gradient of the whole block. A value passes at most 6
    roundings to bf16 (half an ulp, 2^-8 relative, each) on its way, whose
    errors add up to less than 6 2^-8 of the norm."""
    g = torch.Generator()
    g.manual_seed(n + c)
    t = torch.randn(n, c, generator=g).to(torch.bfloat16)
    x = torch.randn(n, c, generator=g).to(torch.bfloat16)
    dout = (torch.randn(n, c, generator=g) * 0.1).to(torch.bfloat16)
    w = block.make_weights(c, hidden, 3)
    w["norm"] = (1 + 0.1 * torch.randn(c, generator=g)).to(torch.bfloat16).cuda()
    w["bias"] = (0.1 * torch.randn(c, generator=g)).to(torch.bfloat16).cuda()
    out, saved = block.forward(t.cuda(), x.cuda(), w)
    ds, grads = block.backward(dout.cuda(), saved, w)

    p = {k: v.cpu().double().requires_grad_(True) for k, v in w.items()}
    td = t.double().requires_grad_(True)
    s = td + x.double()
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + block.EPS) * p["norm"]
    z = y @ p["gated"]
    ref = (ro.act(z[:, :hidden], "silu") * z[:, hidden:]) @ p["down"] + p["bias"] + s
    keys = list(p)
    want = torch.autograd.grad(ref, [td] + [p[k] for k in keys], dout.double())

    def off(a, b):
        return ((a.double().cpu() - b).norm() / b.norm()).item()

    tol = 6 * 2.0 ** -8
    assert off(out, ref.detach()) <= tol
    assert off(ds, want[0]) <= tol
    for k, v in zip(keys, want[1:]):
        assert off(grads[k], v) <= tol, k


def test_example_trains_and_serves(block):
    losses, off = block.main(n=2000, steps=6)
    assert losses[-1] < losses[0]
    # both operands of the gated layer rounded to 3 mantissa bits: at most 2^-4
    # each, on one of two summands of the output
    assert off < 2 * 2.0 ** -4
