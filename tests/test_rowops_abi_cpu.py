"""The row operators' C entries refuse bad arguments before any GPU work: their
host code built with AddressSanitizer and UndefinedBehaviorSanitizer (host pass
only) and driven by a C program. The binding's structures match the header's."""
import ctypes
import os
import re
import subprocess

import pytest

import submanifold_sparse_convolution_amd as smc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "submanifold_sparse_convolution_amd", "csrc")


def test_row_operators_host_code_under_asan_and_ubsan(tmp_path):
    build = os.path.join(ROOT, "_build")
    objs = sorted(f for f in os.listdir(build) if f.endswith(".o")) if os.path.isdir(build) else []
    if "pointwise_api.o" not in objs:
        pytest.fail("the library objects are not built (run __graft_entry__.build())")
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    inc = ["-I", os.path.join(ROOT, "include")]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined"]
    made = []
    for name in ("pointwise_api", "smconv_api"):
        made.append(str(tmp_path / (name + ".o")))
        subprocess.run([hipcc, "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
                        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *san, *inc,
                        "-c", os.path.join(CSRC, name + ".hip"), "-o", made[-1]],
                       check=True, capture_output=True)
    lib = str(tmp_path / "libsmconv_asan.so")
    others = [os.path.join(build, f) for f in objs if f not in ("pointwise_api.o", "smconv_api.o")]
    subprocess.run([hipcc, "-shared", "-fPIC", "--offload-arch=gfx950", *san, *made, *others, "-o", lib],
                   check=True, capture_output=True)
    exe = str(tmp_path / "abi_rowops_check")
    subprocess.run(["/opt/rocm/llvm/bin/clang", "-O1", "-g", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", *inc,
                    os.path.join(ROOT, "tests", "abi_rowops_check.c"), lib,
                    "-Wl,-rpath," + str(tmp_path), "-lm", "-o", exe], check=True, capture_output=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", HIP_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "row operators abi check ok" in r.stdout


@pytest.mark.parametrize("struct,mirror", [("smc_norm_t", smc.NormArgs), ("smc_norm_backward_t", smc.NormBackwardArgs),
                                           ("smc_product_t", smc.ProductArgs)])
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
