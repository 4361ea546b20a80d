"""AddressSanitizer / UndefinedBehaviorSanitizer run, on the CPU, of the host side of moe_lora_linear_lora,
moe_lora_block_norm and moe_lora_forward_few (csrc/api_block.hip): argument checks, plans and workspace sizes,
linked against launchers that abort if reached. Sanitizers apply to host code only."""
import os

import pytest

from tests.test_sanitizers import CLANG, CSRC, ENV, HIPCC, ROOT, SAN, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm toolchain missing")
def test_block_operators_host_checks_under_asan_ubsan(tmp_path):
    host_san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                "-Xarch_host", "-fno-omit-frame-pointer"]
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature",
             "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, *host_san]
    objs = []
    for src in (os.path.join(CSRC, "api_block.hip"), os.path.join(CSRC, "api_ops.hip"),
                os.path.join(SAN, "block_stub_launchers.hip"), os.path.join(SAN, "ops_stub_launchers.hip")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, *flags, "-c", src, "-o", obj])
        objs.append(obj)
    drv = str(tmp_path / "block_host_checks.o")
    _run([CLANG, "-O1", "-g", "-fsanitize=address,undefined", "-fno-omit-frame-pointer",
          "-I" + os.path.join(ROOT, "include"), "-c", os.path.join(SAN, "block_host_checks.c"), "-o", drv])
    exe = str(tmp_path / "block_san")
    _run([HIPCC, "--offload-arch=gfx950", "-fsanitize=address,undefined", "-fno-gpu-sanitize", *objs, drv,
          "-o", exe])
    r = _run([exe], env=ENV, timeout=300)
    assert "ok" in r.stdout
