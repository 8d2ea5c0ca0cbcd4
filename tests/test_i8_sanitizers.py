"""The argument checks of the 8-bit integer calls, the routing and the combination
(csrc/rz_i8_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer, with
stub launchers (csrc/i8_host_check.cpp); CPU only.  The build stops at the first
report, so a clean exit status means no report."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]
CLANG = "/opt/rocm/llvm/bin/clang++"


def test_i8_checks_are_clean_under_asan_and_ubsan(tmp_path):
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang missing")
    exe = str(tmp_path / "i8_hostcheck")
    csrc = os.path.join(ROOT, "nvfp4_razer_w4a16_amd", "csrc")
    for cmd in ([CLANG, "-x", "c++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", *SAN, "-o", exe,
                 os.path.join(csrc, "rz_i8_api.cpp"), os.path.join(csrc, "i8_host_check.cpp"),
                 "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], [exe]):
        r = subprocess.run(cmd, capture_output=True, text=True, cwd=tmp_path)
        assert r.returncode == 0, f"{r.stdout}\n{r.stderr}"
    assert "i8_host_check: ok" in r.stdout
