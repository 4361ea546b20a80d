"""AddressSanitizer / UndefinedBehaviorSanitizer run, on the CPU, of the host side of moe_lora_route and
moe_lora_linear (csrc/api_ops.hip): argument checks, the choice of kernel and workspace sizes, linked
against launchers that abort if reached. Sanitizers apply to host code only."""
import os

import pytest

from tests.test_sanitizers import CLANG, CSRC, ENV, HIPCC, ROOT, SAN, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm toolchain missing")
def test_operators_host_checks_under_asan_ubsan(tmp_path):
    host_san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                "-Xarch_host", "-fno-omit-frame-pointer"]
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature",
             "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, *host_san]
    objs = []
    for src in (os.path.join(CSRC, "api_ops.hip"), os.path.join(SAN, "ops_stub_launchers.hip")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, *flags, "-c", src, "-o", obj])
        objs.append(obj)
    drv = str(tmp_path / "ops_host_checks.o")
    _run([CLANG, "-O1", "-g", "-fsanitize=address,undefined", "-fno-omit-frame-pointer",
          "-I" + os.path.join(ROOT, "include"), "-c", os.path.join(SAN, "ops_host_checks.c"), "-o", drv])
    exe = str(tmp_path / "ops_san")
    _run([HIPCC, "--offload-arch=gfx950", "-fsanitize=address,undefined", "-fno-gpu-sanitize", *objs, drv,
          "-o", exe])
    r = _run([exe], env=ENV, timeout=300)
    assert "ok" in r.stdout


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm toolchain missing")
def test_given_choices_host_checks_under_asan_ubsan(tmp_path):
    """The host side of moe_lora_forward_topk (csrc/api.hip), and adapter counts up to the largest int."""
    host_san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                "-Xarch_host", "-fno-omit-frame-pointer"]
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature",
             "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, *host_san]
    objs = []
    for src in (os.path.join(CSRC, "api.hip"), os.path.join(SAN, "stub_launchers.hip")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, *flags, "-c", src, "-o", obj])
        objs.append(obj)
    drv = str(tmp_path / "topk_host_checks.o")
    _run([CLANG, "-O1", "-g", "-fsanitize=address,undefined", "-fno-omit-frame-pointer",
          "-I" + os.path.join(ROOT, "include"), "-c", os.path.join(SAN, "topk_host_checks.c"), "-o", drv])
    exe = str(tmp_path / "topk_san")
    _run([HIPCC, "--offload-arch=gfx950", "-fsanitize=address,undefined", "-fno-gpu-sanitize", *objs, drv,
          "-o", exe])
    r = _run([exe], env=ENV, timeout=300)
    assert "ok" in r.stdout
