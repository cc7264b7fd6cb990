"""Sanitizer builds of the delta rule's and the group norm's host side (CPU only).

csrc/delta_api.cpp and csrc/norm_api.cpp, compiled with AddressSanitizer + UndefinedBehaviorSanitizer and
separately with ThreadSanitizer, are linked with the library's kernel objects into
tests/sanitize/delta_norm_fuzz.cpp.  Every call it makes returns before a launch, so no GPU is needed.
"""
import os

import pytest

from tests.test_host_sanitizers import CLANG, ROOT, SAN, _kernel_objects, _run


@pytest.mark.parametrize("san", ["address,undefined", "thread"])
def test_delta_and_norm_host_side_under_sanitizers(tmp_path, san):
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang++ not available")
    flags = ["-O1", "-g", "-std=c++17", "-fno-omit-frame-pointer", f"-fsanitize={san}"]
    if san != "thread":
        flags.append("-fno-sanitize-recover=all")
    objs = []
    for name in ("delta_api.cpp", "norm_api.cpp", "convfwd_api.cpp"):
        objs.append(str(tmp_path / (name + ".o")))
        _run([CLANG, *flags, "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-c",
              os.path.join(ROOT, "implicit_gemm_conv_amd", "csrc", name), "-o", objs[-1]])
    main, exe = str(tmp_path / "main.o"), str(tmp_path / "delta_norm_fuzz")
    _run([CLANG, *flags, "-c", os.path.join(SAN, "delta_norm_fuzz.cpp"), "-o", main])
    _run([CLANG, f"-fsanitize={san}", main, *objs, *_kernel_objects(), "-o", exe, "-L/opt/rocm/lib", "-lamdhip64",
          "-lpthread", "-Wl,-rpath,/opt/rocm/lib"])
    env = {**os.environ, "TSAN_OPTIONS": "halt_on_error=1", "ASAN_OPTIONS": "detect_leaks=0"}
    assert "0 inconsistent answers" in _run([exe, "8", "20000"], env=env, timeout=300)
