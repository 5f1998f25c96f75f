"""Argument validation of the attention over the paged cache, compaction, the page pool and rotary positions: a host build of
csrc/draft_api.cpp under AddressSanitizer and UndefinedBehaviorSanitizer with stand-in launchers
(tests/native/drafts_check.cpp)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_validation_under_asan_and_ubsan(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "drafts_check")
    sources = [os.path.join(ROOT, "mixed_precision_moe_amd", "csrc", "draft_api.cpp"),
               os.path.join(ROOT, "tests", "native", "drafts_check.cpp")]
    cmd = [cxx, "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), *sources, "-o", exe]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0 and "draft checks passed" in r.stdout, r.stdout
