"""The C ABI of gdn_glr_*, gdn_rope_* and gdn_swa_* (gdn_hybrid_abi.cpp) under AddressSanitizer
and UndefinedBehaviorSanitizer, CPU only: built with g++ against host stand-ins for the
launchers and driven by tests/sanitize/hybrid_driver.cpp.  Any report aborts the driver."""
import os
import shutil

import pytest

from test_sanitizers import CSRC, ENV, FLAGS, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_hybrid_abi_under_sanitizers(tmp_path):
    exe = str(tmp_path / "hybrid_driver")
    r = _run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
              "-I" + CSRC, *FLAGS, os.path.join(CSRC, "gdn_abi.cpp"), os.path.join(CSRC, "gdn_hybrid_abi.cpp"),
              os.path.join(SAN, "stubs.cpp"), os.path.join(SAN, "hybrid_stubs.cpp"), os.path.join(SAN, "hybrid_driver.cpp"),
              "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    assert r.returncode == 0, r.stderr[-4000:]
    r = _run([exe], env=ENV)
    print(r.stdout[-2000:])
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert r.stdout.strip().splitlines()[-1].startswith("ok:")
