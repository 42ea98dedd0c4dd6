"""Launches, grids and allocations of the decode step's operators, seen by a program that stands
in for the HIP runtime (tests/decode_launches.cpp): no GPU, nothing runs."""
import os
import subprocess

import block_scaled_fp8_token_amd as F
from block_scaled_fp8_token_amd.build import HIPCC

HERE = os.path.dirname(os.path.abspath(__file__))


def test_launches(tmp_path):
    out = str(tmp_path / "decode_launches")
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(rocm, "include"),
                        os.path.join(HERE, "decode_launches.cpp"), "-o", out, "-rdynamic", "-pthread", F.library_path(),
                        "-Wl,-rpath," + os.path.join(rocm, "lib")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
