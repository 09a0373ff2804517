"""The host half of the paged KV cache built under AddressSanitizer and
UndefinedBehaviorSanitizer (g++, CPU only) and driven by a randomised program
in tests/sanitize/ whose device steps act on host memory."""
import os
import shutil
import subprocess

import pytest

from test_sanitizers import ROOT, SAN, _run

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


def test_kv_host_half_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "kv_driver")
    csrc = os.path.join(ROOT, "segmented_gather_gemm_segments_amd", "csrc")
    subprocess.check_call(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                           "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "host.cpp"),
                           os.path.join(csrc, "kv_host.cpp"), os.path.join(ROOT, "tests", "sanitize", "kv_driver.cpp"),
                           "-o", exe])
    assert "kv driver ok" in _run(exe)


def test_kv_marks_that_fail_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "kv_mark_driver")
    csrc = os.path.join(ROOT, "segmented_gather_gemm_segments_amd", "csrc")
    subprocess.check_call(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                           "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "host.cpp"),
                           os.path.join(csrc, "kv_host.cpp"), os.path.join(ROOT, "tests", "sanitize", "kv_mark_driver.cpp"),
                           "-o", exe])
    assert "kv mark driver ok" in _run(exe)
