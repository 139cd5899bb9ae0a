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
