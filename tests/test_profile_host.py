"""The timing facility's readers write a caller's arrays up to their length and
no further (``tests/host/profile_check.cpp``, built with g++)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_cross_entropy_gemm_amd", "csrc")


def test_profile_readers_keep_to_the_callers_arrays(tmp_path):
    gxx = shutil.which("g++")
    if not gxx or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("g++ and the ROCm headers are needed")
    exe = str(tmp_path / "profile_check")
    subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I",
                    os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(ROOT, "tests", "host", "profile_check.cpp"),
                    os.path.join(CSRC, "flce_profile.cpp"), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "0 failed checks\n", r.stdout
