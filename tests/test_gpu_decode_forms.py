"""The operators of a decode step in every form that their sizes choose: values against references in 64 bits and values that
are not finite (tests/test_decode_forms.py checks that no kernel is left out)."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_token_amd as F
import test_gpu_decode_ops as ops
from test_gpu_decode_ops import DEV, FORMATS, KINDS, bf16, weights_of

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


@pytest.mark.parametrize("format,group,zero_points", FORMATS)
@pytest.mark.parametrize("T,N,K", [
    # one tile a wavefront, several units of 512 columns and a part of one for each
    (1, 48, 7296), (4, 100, 6784), (7, 48, 6784), (12, 31, 7296), (17, 48, 6784), (33, 100, 7296), (64, 40, 4224),
    (130, 33, 3200),
    # two tiles
    (2, 5152, 4224), (11, 4112, 3200), (20, 4112, 3200), (40, 4112, 2688), (64, 4112, 2176),
    # tokens through LDS, several chunks of them for each half of K
    (5, 8224, 4224), (20, 8300, 3200), (40, 8400, 1664), (64, 8210, 1664), (9, 16400, 2688), (36, 16390, 1152)])
def test_gemv(format, group, zero_points, T, N, K):
    """Products whose wavefronts take several turns over K, of columns that are no multiple of 512."""
    ops.test_gemv(format, group, zero_points, T, N, K)


@pytest.mark.parametrize("format,group,zero_points", FORMATS)
@pytest.mark.parametrize("T,N", [(3, 100), (7, 5152), (14, 40), (20, 48), (40, 4128), (60, 100), (20, 8300), (60, 16400),
                                 (70, 100)])
def test_gemv_values_that_are_not_finite_stay_with_their_token(format, group, zero_points, T, N):
    """With four, two and one K-blocks of the tokens side by side, with several blocks of tokens, and through LDS."""
    rng = np.random.default_rng([T, N, group])
    K = 640
    _, _, laid = weights_of(rng, N, K, format, group, zero_points)
    x = bf16(rng, T, K)
    clean = F.w4_group_gemv_nt(x.to(DEV), laid[0], laid[1], N, zeros=laid[2])
    x[1, K - 1] = float("nan")
    x[T - 1, 130] = float("inf")
    got = F.w4_group_gemv_nt(x.to(DEV), laid[0], laid[1], N, zeros=laid[2])
    same = [t for t in range(T) if t not in (1, T - 1)]
    assert clean.isfinite().all() and torch.equal(got[same], clean[same])
    assert got[1].isnan().all() and not got[T - 1].isfinite().any()
