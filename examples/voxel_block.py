"""A residual block on active voxels: sparse convolution, then the row operators.

    t = conv(x)                              27-tap submanifold convolution
    y, s = rms_norm(t, residual=x)           s = t + x, the new residual stream
    h = gated(y)                             silu(y Wg) * (y Wu)
    out = linear(h, residual=s)              h Wd + b + s

Run on a GPU (`python examples/voxel_block.py`): a few training steps of the
block's own weights against a random target, then the trained block served in
16 bits and in e4m3, whose outputs are compared.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import submanifold_sparse_convolution_amd as smc  # noqa: E402
import synth  # noqa: E402

EPS = 1e-6


def make_weights(c, hidden, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    return dict(norm=torch.ones(c, dtype=dtype, device="cuda"),
                gated=normal(c, 2 * hidden, std=c ** -0.5),
                down=normal(hidden, c, std=hidden ** -0.5),
                bias=torch.zeros(c, dtype=dtype, device="cuda"))


def forward(t, x, w):
    """The block behind the convolution's output t and the residual stream x:
    (out, what the backward pass needs)."""
    y, s = smc.rms_norm(t, w["norm"], residual=x, eps=EPS)
    h = smc.gated(y, w["gated"])
    out = smc.linear(h, w["down"], bias=w["bias"], residual=s)
    return out, (y, s, h)


def backward(dout, saved, w):
    """(gradient of t and of x alike, gradients of the weights)."""
    y, s, h = saved
    dh, ddown, dbias = smc.linear_backward(dout, h, w["down"], bias=w["bias"])
    dy, dgated, _ = smc.gated_backward(dh, y, w["gated"])
    # out takes s twice: through the norm, and as the residual
    ds, dnorm = smc.rms_norm_backward(dy, s, w["norm"], eps=EPS, ds=dout)
    return ds, dict(norm=dnorm, gated=dgated, down=ddown, bias=dbias)


def quantise(w):
    """The weights of the 8-bit block, made once."""
    return dict(w, gated=smc.quantize_weight(w["gated"]))


def forward_e4m3(t, x, w):
    """forward with the gated layer on e4m3 rows."""
    q, scale, s = smc.rms_norm(t, w["norm"], residual=x, eps=EPS, e4m3=True)
    wq, w_scale = w["gated"]
    h = smc.gated(q, wq, x_scale=scale, w_scale=w_scale, dtype=t.dtype)
    return smc.linear(h, w["down"], bias=w["bias"], residual=s)


def main(n=8000, c=64, hidden=176, steps=8, lr=2.0):
    grid = (128, 128, 24)
    g = torch.Generator()
    g.manual_seed(0)
    cells = torch.randperm(grid[0] * grid[1] * grid[2], generator=g)[:n]
    coords = torch.stack((cells // (grid[1] * grid[2]), cells // grid[2] % grid[1], cells % grid[2]), 1)
    bits = torch.from_numpy(synth.features(n, c, 1).view("int16"))
    x = bits.view(torch.bfloat16).cuda()
    wconv = torch.from_numpy(synth.weights(c, c, 1).view("int16")).view(torch.bfloat16).cuda()
    m = smc.KernelMap().build(coords.int().cuda(), spatial_shape=grid)
    t = m.forward(x, smc.pack_weights(wconv))
    target = torch.randn(n, c, generator=g).cuda()

    w = make_weights(c, hidden, 1)
    master = {k: v.float() for k, v in w.items()}
    losses = []
    for _ in range(steps):
        out, saved = forward(t, x, w)
        diff = out.float() - target
        losses.append((diff ** 2).mean().item())
        _, grads = backward((diff * (2.0 / diff.numel())).to(out.dtype), saved, w)
        for k in w:
            master[k] -= lr * grads[k].float()
            w[k] = master[k].to(out.dtype)
    a = forward(t, x, w)[0].float()
    b = forward_e4m3(t, x, quantise(w)).float()
    off = ((a - b).norm() / a.norm()).item()
    m.close()
    print("loss", " ".join(f"{v:.4f}" for v in losses), f"| e4m3 against 16 bits: {off:.4f} of the norm")
    return losses, off


if __name__ == "__main__":
    main()
