"""The host code of the third part of the C ABI (include/mxfp4.h: validation and
the grid helpers behind it) under AddressSanitizer + UndefinedBehaviorSanitizer,
driven with extreme sizes by tests/sanitize/fp4_driver.cpp.  Host code only: the
kernels are built without a sanitizer and never run."""
import os

import pytest

from tests.test_sanitizers import CSRC, ENV, HERE, HIPCC, OUT, ROOT, _run


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is present; this build runs where none is")
def test_fp4_host_code_under_asan_ubsan():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not found")
    os.makedirs(OUT, exist_ok=True)
    exe = os.path.join(OUT, "fp4_asan")
    srcs = [os.path.join(CSRC, f) for f in ("mx_fp4_api.hip", "mx_fp4_cast.hip", "mx_mm_gemm.hip", "mx_mm_ffn.hip",
                                           "mx_decode.hip")]
    b = _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fno-omit-frame-pointer",
              "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
              "-Xarch_host", "-fno-sanitize-recover=all",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-I", os.path.join(ROOT, "include"), "-I", CSRC, *srcs, os.path.join(HERE, "fp4_driver.cpp"), "-o", exe])
    assert b.returncode == 0, b.stderr[-4000:]
    r = _run([exe], env=ENV, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "runtime error" not in r.stderr and "ERROR: AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert "fp4 sanitizer run clean" in r.stdout
