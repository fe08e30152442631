"""The operators' overlap check against a byte-by-byte answer, built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer (tests/sanitize/overlap.cpp).  CPU only."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ring_allreduce_reduction_amd", "csrc")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]


def test_overlap_check_against_bytes(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path / "overlap")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run(["g++", "-std=c++17", "-Wall"] + SAN + ["-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I",
                   os.path.join(rocm, "include"), os.path.join(CSRC, "ar_api.cpp"),
                   os.path.join(ROOT, "tests", "sanitize", "overlap.cpp"), "-o", exe,
                   "-L" + os.path.join(rocm, "lib"), "-Wl,-rpath," + os.path.join(rocm, "lib"),
                   "-lrocprofiler-sdk-roctx"], check=True)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout + p.stderr[-2000:]
