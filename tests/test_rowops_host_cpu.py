"""Host rules of the row operators that need no GPU: overlapping buffers and the
sizes of scratch memory. The addresses below are never read: a call that passes
the argument checks ends at the missing device."""
import os
import subprocess
import sys

import pytest

import submanifold_sparse_convolution_amd as smc

SMC_ERR_ARG = 1
BASE = 1 << 20


def norm(**kw):
    a = smc.NormArgs(8, 64, 0, 1e-6, BASE, 64, None, 0, BASE << 4, BASE << 5, 64, BASE << 6, None, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


# y e4m3 (one byte an element) against x, residual and s (two bytes): 8 rows of 64
SHARED = [
    dict(y=BASE),                                               # row r of y over row r / 2 of x
    dict(y=BASE, ldy=128),                                      # equal distances in bytes
    dict(y=BASE + 64, ldy=128),                                 # the second half of each row of x
    dict(y=BASE + 8 * 128 - 1),                                 # the last byte of x
    dict(y=BASE - 8 * 64 + 1),                                  # y's last byte
    dict(residual=BASE << 5, ld_residual=64),
    dict(s=BASE << 5, lds=64),
]
APART = [
    dict(y=BASE + 8 * 128),                                     # right after x
    dict(y=BASE - 8 * 64),                                      # right before it
    dict(y=BASE + 128, ldy=256, ldx=128),                       # columns of one buffer
    dict(y=BASE - 64, ldy=256, ldx=128),
    dict(residual=BASE, ld_residual=64, s=BASE, lds=64),        # in place, y elsewhere
]


# outputs of the layers over inputs that other blocks, or later kernels, still read
W, Y, DY, DX, FAR = (BASE << k for k in range(1, 6))


def product(**kw):
    a = smc.ProductArgs(8, 64, 64, 0, 0, 0, BASE, 64, None, W, 128)
    a.y, a.ldy, a.dy, a.ld_dy, a.dx, a.ld_dx, a.dw, a.ld_dw = Y, 64, DY, 64, DX, 64, FAR, 128
    a.workspace, a.workspace_bytes = FAR << 1, 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return a


LAYERS, BACK = ("smc_linear", "smc_gated"), ("smc_linear_backward", "smc_gated_backward")
OVER = ([(name, dict(y=BASE)) for name in LAYERS] + [(name, dict(y=BASE + 128 * 8 - 2)) for name in LAYERS]
        + [(name, dict(dx=BASE)) for name in BACK] + [("smc_linear_backward", dict(dx=DY))]
        + [("smc_linear", dict(x_dtype=2, x_scale=FAR, w_scale=FAR, y=BASE))])
BESIDE = ([(name, dict(y=BASE + 128, ldy=128, ldx=128)) for name in LAYERS]
          + [("smc_linear", dict(residual=Y, ld_residual=64))]
          + [("smc_linear_backward", dict(dx=DY + 128, ld_dx=128, ld_dy=128))])
CALLS = [("smc_rms_norm", kw) for kw in SHARED + APART] + OVER + BESIDE


@pytest.fixture(scope="module")
def answers():
    """Status and message of every call, from a process that sees no device (and
    makes no call if it does)."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = %r\n"
            "import ctypes, torch, test_rowops_host_cpu as t\n"
            "import submanifold_sparse_convolution_amd as smc\n"
            "assert torch.cuda.device_count() == 0\n"
            "for name, kw in t.CALLS:\n"
            "    args = t.norm(**kw) if name == 'smc_rms_norm' else t.product(**kw)\n"
            "    rc = getattr(smc.lib(), name)(ctypes.byref(args), None)\n"
            "    print(rc, smc.lib().smc_last_error().decode())\n" % [here, os.path.dirname(here)])
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1")
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    lines = out.stdout.strip().splitlines()
    assert len(lines) == len(CALLS)
    return [(int(line.partition(" ")[0]), line.partition(" ")[2]) for line in lines]


@pytest.mark.parametrize("i", range(len(SHARED)))
def test_e4m3_rows_that_share_memory_are_refused(answers, i):
    rc, msg = answers[i]
    assert rc == SMC_ERR_ARG and "shares memory" in msg, (SHARED[i], rc, msg)


@pytest.mark.parametrize("i", range(len(APART)))
def test_e4m3_rows_beside_the_inputs_pass_the_checks(answers, i):
    rc, msg = answers[len(SHARED) + i]
    assert rc != SMC_ERR_ARG, (APART[i], rc, msg)


@pytest.mark.parametrize("i", range(len(OVER)))
def test_layers_over_their_inputs_are_refused(answers, i):
    rc, msg = answers[len(SHARED) + len(APART) + i]
    assert rc == SMC_ERR_ARG and "shares memory" in msg, (OVER[i], rc, msg)


@pytest.mark.parametrize("i", range(len(BESIDE)))
def test_layers_beside_their_inputs_pass_the_checks(answers, i):
    rc, msg = answers[len(SHARED) + len(APART) + len(OVER) + i]
    assert rc != SMC_ERR_ARG, (BESIDE[i], rc, msg)


@pytest.mark.parametrize("n,c_in,c_out", [(1, 8, 8), (257, 8, 8), (15000, 2048, 512), (15000, 512, 4096),
                                          (91000, 128, 688), (95000, 144, 256), (131584, 128, 128),
                                          (1000000, 64, 64), (300, 3000, 3104)])
def test_every_range_of_a_weight_gradient_has_rows(n, c_in, c_out):
    """Aligned operands and no activation: the scratch memory holds the ranges' sums
    alone. A range is a multiple of 64 rows; the last one begins before row n."""
    a = smc.ProductArgs(n, c_in, c_out, 0, 0, 0, BASE, c_in, None, BASE, c_out)
    a.dy, a.ld_dy, a.dx, a.ld_dx, a.dw, a.ld_dw = BASE, c_out, BASE, c_in, BASE, c_out
    ranges, rest = divmod(smc.lib().smc_linear_backward_workspace(a), c_in * c_out * 4)
    assert ranges >= 1 and rest == 0
    length = -(-(-(-n // ranges)) // 64) * 64
    assert (ranges - 1) * length < n, f"{ranges} ranges of {length} rows for {n}"


@pytest.mark.parametrize("n,c,rows_a_block", [(1, 128, 16), (1000, 128, 16), (1000, 7, 256), (1000, 257, 4),
                                              (37, 4096, 4), (1000, 4097, 1), (95000, 128, 16)])
def test_every_block_of_a_norm_gradient_has_rows(n, c, rows_a_block):
    """The scratch memory is one row of sums a block (rounded up to 256 bytes):
    no more blocks than the rows need, 256 threads each, or than 4 a CU."""
    blocks = min(-(-n // rows_a_block), 4 * 256)
    assert smc.lib().smc_rms_norm_backward_workspace(n, c) == -(-blocks * c * 4 // 256) * 256
