"""What the host code of the entry points launches, allocates and waits for, seen by a program
that stands in for the HIP runtime (tests/host_launches.cpp): no GPU, nothing runs."""
import os
import subprocess

import pytest

import block_scaled_fp8_token_amd as F
from block_scaled_fp8_token_amd.build import HIPCC

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("host") / "host_launches")
    # -rdynamic: the program's definitions of the runtime's functions are the ones the library finds
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(rocm, "include"),
                        os.path.join(HERE, "host_launches.cpp"), "-o", out, "-rdynamic", "-pthread", F.library_path(),
                        "-Wl,-rpath," + os.path.join(rocm, "lib")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return out


def run(program, scenario):
    r = subprocess.run([program, scenario], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


def test_threads_on_one_stream(program):
    run(program, "threads")


def test_threads_on_the_scratch_of_the_entry_that_allocates_nothing(program):
    run(program, "noalloc_threads")


def test_largest_sizes(program):
    run(program, "limits")


def test_combine_backward_without_columns(program):
    run(program, "no_columns")


def test_norm_backward_of_one_row_allocates_nothing(program):
    run(program, "one_row")


def test_norm_backward_in_scratch_of_the_callers(program):
    run(program, "given_scratch")
