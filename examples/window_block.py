"""A residual block of windowed attention on active voxels, behind a sparse convolution.

    t = conv(x)                                       27-tap submanifold convolution
    y = silu(group_norm(t))                           over the rows of each sample
    q, k, v = columns of linear(y)                    one projection
    a = window_attention(q, k, v)                     inside windows of 8 x 8 x 8 voxels, with a learned
                                                      bias by relative position
    out = linear(a, residual=x)                       a Wo + b + x

Run on a GPU (`python examples/window_block.py`): a few training steps of the block's own
weights against a random target.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import submanifold_sparse_convolution_amd as smc  # noqa: E402

SIZE = 8                # a window's cells along each axis
GROUPS, HEADS = 8, 4


def make_windows(coords, shift=0):
    """The windows of SIZE^3 cells that hold the rows of int32 [N, 4] (b, x, y, z) coordinates, the grid of
    windows moved by `shift` cells (every other block takes SIZE / 2, so that neighbours meet)."""
    cell = torch.cat((coords[:, :1], (coords[:, 1:] + shift) // SIZE), 1).long()
    wide = cell.amax(0) + 1
    key = ((cell[:, 0] * wide[1] + cell[:, 1]) * wide[2] + cell[:, 2]) * wide[3] + cell[:, 3]
    key, order = torch.sort(key, stable=True)
    counts = torch.unique_consecutive(key, return_counts=True)[1]
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0))).int()
    return smc.Windows(offsets, len(coords), order=order.int(), coords=coords, extent=(SIZE,) * 3)


def sample_offsets(coords, samples):
    """Where each sample's rows begin (rows sorted by sample)."""
    return torch.searchsorted(coords[:, 0].contiguous(), torch.arange(samples + 1, device=coords.device,
                                                                     dtype=torch.int32)).int()


def make_weights(c, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def full(value, *shape):
        return torch.full(shape, value, dtype=dtype, device="cuda")

    return dict(norm=full(1.0, c), norm_bias=full(0.0, c), qkv=normal(c, 3 * c, std=c ** -0.5), qkv_bias=full(0.0, 3 * c),
                table=normal(3, 2 * SIZE - 1, HEADS, std=0.02), out=normal(c, c, std=c ** -0.5), out_bias=full(0.0, c))


def forward(t, x, w, windows, offsets):
    """The block behind the convolution's output t and the residual stream x: (out, what the backward
    pass needs)."""
    y, stats = smc.group_norm(t, w["norm"], w["norm_bias"], GROUPS, offsets=offsets, activation="silu", stats=True)
    qkv = smc.linear(y, w["qkv"], bias=w["qkv_bias"])
    q, k, v = qkv.chunk(3, 1)
    a, lse = smc.window_attention(q, k, v, windows, HEADS, bias=w["table"], lse=True)
    out = smc.linear(a, w["out"], bias=w["out_bias"], residual=x)
    return out, (t, stats, y, qkv, a, lse)


def backward(dout, saved, w, windows, offsets):
    """(gradient of t, gradients of the weights); the gradient of x is dout."""
    t, stats, y, qkv, a, lse = saved
    da, dout_w, dout_b = smc.linear_backward(dout, a, w["out"], bias=w["out_bias"])
    dqkv = torch.empty_like(qkv)
    _, _, _, dtable = smc.window_attention_backward(da, *qkv.chunk(3, 1), a, lse, windows, HEADS, bias=w["table"],
                                                    grads=dqkv.chunk(3, 1))
    dy, dqkv_w, dqkv_b = smc.linear_backward(dqkv, y, w["qkv"], bias=w["qkv_bias"])
    dt, dnorm, dnorm_b = smc.group_norm_backward(dy, t, w["norm"], w["norm_bias"], GROUPS, stats, offsets=offsets,
                                                 activation="silu")
    return dt, dict(norm=dnorm, norm_bias=dnorm_b, qkv=dqkv_w, qkv_bias=dqkv_b, table=dtable, out=dout_w, out_bias=dout_b)


def make_cells(n, samples, grid, seed):
    """n voxels of `samples` grids, sorted by sample, int32 [n, 4]."""
    g = torch.Generator()
    g.manual_seed(seed)
    volume = grid[0] * grid[1] * grid[2]
    cells = torch.randperm(samples * volume, generator=g)[:n].sort().values
    b, cells = cells // volume, cells % volume
    return torch.stack((b, cells // (grid[1] * grid[2]), cells // grid[2] % grid[1], cells % grid[2]), 1).int().cuda()


def main(n=8000, c=64, steps=8, lr=0.5):
    grid, samples = (64, 64, 16), 2
    coords = make_cells(n, samples, grid, 0)
    g = torch.Generator()
    g.manual_seed(1)
    x = torch.randn(n, c, generator=g).to(torch.bfloat16).cuda()
    wconv = (torch.randn(27, c, c, generator=g) * (27 * c) ** -0.5).to(torch.bfloat16).cuda()
    target = torch.randn(n, c, generator=g).cuda()
    m = smc.KernelMap().build(coords, spatial_shape=grid, batch_size=samples)
    t = m.forward(x, smc.pack_weights(wconv))
    windows, offsets = make_windows(coords), sample_offsets(coords, samples)

    w = make_weights(c, 2)
    master = {k: v.float() for k, v in w.items()}
    losses = []
    for _ in range(steps):
        out, saved = forward(t, x, w, windows, offsets)
        diff = out.float() - target
        losses.append((diff ** 2).mean().item())
        _, grads = backward((diff * (2.0 / diff.numel())).to(out.dtype), saved, w, windows, offsets)
        for k in w:
            master[k] -= lr * grads[k].float()
            w[k] = master[k].to(out.dtype)
    m.close()
    print("loss", " ".join(f"{v:.4f}" for v in losses), f"| {n} voxels, longest window {windows.longest}")
    return losses


if __name__ == "__main__":
    main()
