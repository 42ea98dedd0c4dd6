"""The operators of a decode step in every form that their sizes choose: values against references
in 64 bits (tests/test_decode_forms.py checks that no kernel is left out)."""
import pytest

import test_gpu_decode_ops as ops
from test_gpu_decode_ops import KINDS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,topk,K,H,base", [
    # up to 16 tokens with more than 64 pairs: routing and tokens of the gate_up product in LDS, 16 or 32 output columns
    (16, 32, 8, 512, 256, True), (16, 8, 5, 4224, 128, False),
    # up to 64 pairs whose y is too large for every workgroup to quantize, 32 output columns
    (16, 4, 4, 4224, 640, True), (13, 6, 4, 4224, 640, False),
    # 17 to 32 tokens, more than 64 pairs, 32 output columns
    (20, 12, 6, 4224, 128, True),
    # as many choices as there may be
    (2, 64, 64, 256, 128, False), (64, 200, 64, 128, 128, True), (3, 1024, 63, 128, 128, False),
    # K in two parts of one and two units of 512, and of two and three, with several tokens an expert
    (2, 16, 8, 1152, 1024, True), (16, 48, 4, 2176, 256, False)])
def test_layer(kind, T, E, topk, K, H, base):
    ops.test_layer(kind, T, E, topk, K, H, base)
