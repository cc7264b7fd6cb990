"""The ranges of memory that the gated delta rule's kernels may touch, checked on the host (CPU only).

tests/sanitize/delta_ranges.cpp includes csrc/delta_params.h, from which the kernels take these ranges too.
"""
import os

import pytest

from tests.test_host_sanitizers import CLANG, SAN, _run


def test_ranges_end_with_their_tensors(tmp_path):
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang++ not available")
    exe = str(tmp_path / "delta_ranges")
    _run([CLANG, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
          "-I/opt/rocm/include", os.path.join(SAN, "delta_ranges.cpp"), "-o", exe, "-L/opt/rocm/lib", "-lamdhip64",
          "-Wl,-rpath,/opt/rocm/lib"])
    assert "0 wrong ranges" in _run([exe], env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
