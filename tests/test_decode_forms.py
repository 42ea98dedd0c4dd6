"""No kernel of the decode step's operators is without a test of its values and of the ways of calling it: the sizes of the
GPU tests, put through the library's own choice of kernels (tests/decode_forms.cpp, which stands in for the HIP runtime;
nothing runs on a GPU)."""
import os
import subprocess

import pytest

import block_scaled_fp8_token_amd as F
import test_gpu_decode_forms as forms
import test_gpu_decode_ops as ops
from block_scaled_fp8_token_amd.build import HIPCC

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def kernels_of(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("forms") / "decode_forms")
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(rocm, "include"),
                        os.path.join(HERE, "decode_forms.cpp"), "-o", out, "-rdynamic", "-pthread", F.library_path(),
                        "-Wl,-rpath," + os.path.join(rocm, "lib")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr

    def of(lines):
        r = subprocess.run([out], input="\n".join(lines), capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout + r.stderr
        return set(r.stdout.splitlines())
    return of


def sizes(*tests):
    """The sizes that tests are parametrised over."""
    return [case for t in tests for mark in t.pytestmark
            if mark.name == "parametrize" and mark.args[0].startswith("T,") for case in mark.args[1]]


def layer(kind, T, topk, E, K, H):
    return "layer %s %d %d %d %d %d" % (kind, T, topk, E, K, H)


def product(format, T, N, K):
    return "product %d %d %d %s %d %d" % (T, N, K, *format)


LAYER = ("moe_gate_up_kernel", "moe_down_kernel")
PRODUCT = ("w4_gemv_kernel", "w4_batch_kernel")


@pytest.mark.parametrize("names,lines", [
    (LAYER, [layer(kind, T, topk, E, K, H) for kind in ops.KINDS
             for T, E, topk, K, H, _ in sizes(ops.test_layer, forms.test_layer)]),
    (LAYER, [layer(kind, *size) for kind in ops.KINDS for size in forms.LAYER_FORMS]),
    (PRODUCT, [product(format, *size) for format in ops.FORMATS
               for size in sizes(ops.test_gemv, ops.test_gemv_of_many_rows, forms.test_gemv)]),
], ids=["layer-values", "layer-calls", "product-values"])
def test_no_kernel_is_left_out(kernels_of, names, lines):
    have = {k for k in kernels_of(["kernels"]) if any(n in k for n in names)}
    missing = have - kernels_of(lines)
    assert have and not missing, "\n".join(sorted(missing))


def test_every_form_of_a_product_is_called(kernels_of):
    """Each choice of tiles and tokens, in one format at least."""
    def form(kernel):
        head, args = kernel.split("<", 1)
        return head.split("::")[-1], args.split(",", 2)[2]
    have = {form(k) for k in kernels_of(["kernels"]) if any(n in k for n in PRODUCT)}
    lines = [product(ops.FORMATS[i % len(ops.FORMATS)], T, N, 640) for i, (T, N) in enumerate(forms.GEMV_FORMS)]
    assert have == {form(k) for k in kernels_of(lines)}
