"""The check of outputs against inputs (csrc/byte_ranges.h), on the CPU against a map of the bytes."""
import shutil

import pytest

from tests.test_sanitizers import CSRC, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_overlap_matches_a_map_of_the_bytes(tmp_path):
    exe = str(tmp_path / "byte_ranges")
    _run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover", "-I" + CSRC,
          SAN + "/byte_ranges_checks.cpp", "-o", exe])
    assert "ok" in _run([exe], timeout=300).stdout
