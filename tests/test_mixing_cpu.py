"""Group norm and window attention without a GPU: refusals under sanitizers, the
binding's structures, and the 64-bit formulas that the GPU tests compare with
(tests/_mixing.py), their gradients checked by differences."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import _mixing as mx
import submanifold_sparse_convolution_amd as smc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "submanifold_sparse_convolution_amd", "csrc")


def test_host_code_under_asan_and_ubsan(tmp_path):
    build = os.path.join(ROOT, "_build")
    objs = sorted(f for f in os.listdir(build) if f.endswith(".o")) if os.path.isdir(build) else []
    if "mixing_api.o" not in objs:
        pytest.fail("the library objects are not built (run __graft_entry__.build())")
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    inc = ["-I", os.path.join(ROOT, "include")]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined"]
    made = []
    for name in ("mixing_api", "smconv_api"):
        made.append(str(tmp_path / (name + ".o")))
        subprocess.run([hipcc, "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
                        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *san, *inc,
                        "-c", os.path.join(CSRC, name + ".hip"), "-o", made[-1]],
                       check=True, capture_output=True)
    lib = str(tmp_path / "libsmconv_asan.so")
    others = [os.path.join(build, f) for f in objs if f not in ("mixing_api.o", "smconv_api.o")]
    subprocess.run([hipcc, "-shared", "-fPIC", "--offload-arch=gfx950", *san, *made, *others, "-o", lib],
                   check=True, capture_output=True)
    exe = str(tmp_path / "abi_mixing_check")
    subprocess.run(["/opt/rocm/llvm/bin/clang", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", *inc,
                    os.path.join(ROOT, "tests", "abi_mixing_check.c"), lib,
                    "-Wl,-rpath," + str(tmp_path), "-lm", "-o", exe], check=True, capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", HIP_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "mixing operators abi check ok" in r.stdout


@pytest.mark.parametrize("struct,mirror", [("smc_group_norm_t", smc.GroupNormArgs), ("smc_windows_t", smc.WindowsArgs),
                                           ("smc_attention_t", smc.AttentionArgs)])
def test_structures_match_the_header(struct, mirror, tmp_path):
    """Names in order, sizes and offsets (by a C program)."""
    text = open(os.path.join(ROOT, "include", "smconv.h")).read()
    body = re.search(r"typedef struct \w+ \{([^}]*)\} " + struct + ";", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = []
    for decl in body.split(";"):
        if decl.strip():
            names += [re.sub(r".*[\s*]", "", v.strip()) for v in decl.split(",")]
    assert names == [f[0] for f in mirror._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"smconv.h\"\nint main(void) {\n"
                   + "".join(f'    printf("%zu\\n", offsetof({struct}, {n}));\n' for n in names)
                   + f'    printf("%zu\\n", sizeof({struct}));\n    return 0;\n}}\n')
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    out = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert out == [getattr(mirror, n).offset for n in names] + [ctypes.sizeof(mirror)]


@pytest.mark.parametrize("n,c,groups,offsets", [(0, 8, 2, None), (1, 512, 32, None), (91000, 128, 16, 7),
                                                (95000, 128, 32, 3), (15000, 512, 32, 9), (2 ** 31 - 1024, 8, 1, None),
                                                (3, 8192, 4096, 5), (10, 1, 1, 65)])
def test_scratch_of_a_group_norm(n, c, groups, offsets):
    """Two floats a piece and group, and in the backward pass a channel (each part rounded up to 256
    bytes): no more pieces than two a compute unit, and one more for each sample's border."""
    a = smc.GroupNormArgs(n, c, groups, 1 if offsets is None else offsets - 1, 0, 0, 1e-5, None if offsets is None else 1 << 20)
    ahead = smc.lib().smc_group_norm_workspace(a)
    back = smc.lib().smc_group_norm_backward_workspace(a)
    pieces = ahead // (groups * 8)
    assert 1 <= pieces <= 2 * 256 + (0 if offsets is None else offsets + 1) + 256 // (groups * 8)
    assert (back - ahead) // (c * 8) <= pieces + 256 // (c * 8) + 1


# ---- the formulas' gradients by differences -----------------------------------------------
# Central differences in 64 bits at h = 2^-17: an error of order h^2 and of order 2^-52 / h relative to
# values near 1, both below 2^-30; the tolerance is 2^-24 of the gradients' largest.

H, TOL = 2.0 ** -17, 2.0 ** -24


def differences(f, t, probes):
    out = []
    for i in probes:
        up, down = t.clone(), t.clone()
        up.view(-1)[i] += H
        down.view(-1)[i] -= H
        out.append(((f(up) - f(down)) / (2 * H)).item())
    return torch.tensor(out, dtype=torch.float64)


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_group_norm_formulas(name):
    g = torch.Generator()
    g.manual_seed(1)
    n, c, groups, offsets = 13, 12, 3, [1, 5, 5, 12]
    x, dy = (torch.randn(n, c, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(c, generator=g, dtype=torch.float64) for _ in range(2))
    mean, rstd, _, _ = mx.group_stats(x, groups, offsets, 1e-3)
    stats = torch.stack((mean, rstd), 2)
    got = [t for t, _ in mx.group_norm_backward(dy, x, w, b, groups, stats, offsets, name, torch.bfloat16)]

    def loss(x=x, w=w, b=b):
        return (mx.group_norm(x, w, b, groups, offsets, 1e-3, name, torch.bfloat16)[0] * dy).sum()

    for grad, t, f in ((got[0], x, lambda t: loss(x=t)), (got[1], w, lambda t: loss(w=t)), (got[2], b, lambda t: loss(b=t))):
        probes = range(0, t.numel(), max(1, t.numel() // 40))
        want = differences(f, t, probes)
        assert (grad.reshape(-1)[list(probes)] - want).abs().max() <= TOL * max(1.0, want.abs().max())


@pytest.mark.parametrize("kv", [4, 2])
@pytest.mark.parametrize("table", [False, True])
def test_attention_formulas(kv, table):
    g = torch.Generator()
    g.manual_seed(2)
    n, heads, dim, offsets = 17, 4, 5, [2, 3, 3, 10, 16]
    order = torch.randperm(n, generator=g)
    q, dout = (torch.randn(n, heads * dim, generator=g, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(n, kv * dim, generator=g, dtype=torch.float64) for _ in range(2))
    coords = torch.randint(0, 5, (n, 3), generator=g)
    t = torch.randn(3, 5, heads, generator=g, dtype=torch.float64) if table else None
    rest = (offsets, order, coords if table else None)
    got = [x for x, _ in mx.attention_backward(dout, q, k, v, *rest, t, heads, kv, 0.4, torch.bfloat16)]

    def loss(q=q, k=k, v=v, t=t):
        return (mx.attention(q, k, v, *rest, t, heads, kv, 0.4, torch.bfloat16)[0] * dout).sum()

    pairs = [(q, lambda x: loss(q=x)), (k, lambda x: loss(k=x)), (v, lambda x: loss(v=x))]
    if table:
        pairs.append((t, lambda x: loss(t=x)))
    for grad, (x, f) in zip(got, pairs):
        probes = range(0, x.numel(), max(1, x.numel() // 40))
        want = differences(f, x, probes)
        assert (grad.reshape(-1)[list(probes)] - want).abs().max() <= TOL * max(1.0, want.abs().max())
