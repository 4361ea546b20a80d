"""The check of outputs against inputs (csrc/byte_ranges.h), on the CPU against a map of the bytes."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_overlap_matches_a_map_of_the_bytes(tmp_path):
    exe = str(tmp_path / "byte_ranges")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "lora_mixture_experts_amd", "csrc"),
                    os.path.join(ROOT, "tests", "sanitize", "byte_ranges_checks.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr
