"""The operators of a decode step: a whole mixture-of-experts layer for a few tokens, and
products of a few rows with weights of 4 bits under group scales.

Binding of the entry points of the same names in include/fp8bs.h (which states the
formulas and the layouts).  Checks, streams and values are those of block_ops: wrong types,
shapes and strides raise TypeError or ValueError before anything is launched, all tensors of
a call lie on the current device, nothing is recorded for automatic differentiation, and
outputs that a caller passes must not overlap inputs (not checked).
"""
from __future__ import annotations

import operator

import torch

from . import _lib, _words
from .block_ops import (
    _2d, _BF16, _E4M3, _F32, _I32, _U32, _beside, _launch, _on_stream, _out, _out_rows, _rows, _typed, _whole,
)

__all__ = [
    "moe_decode_layer", "moe_decode_layer_preshuffled", "moe_decode_layer_w4", "w4_group_quant", "w4_preshuffle",
    "w4_group_gemv_nt",
]

_U8 = (torch.uint8,)
_FORMAT = {"e2m1": 0, "int4": 1}


def _moe(name, q, sf, topk_ids, weights, w13, s13, w2, s2, H, shapes, dtypes, base, out):
    T, K = _2d(q, "q")
    topk = _2d(topk_ids, "topk_ids")[1]
    if T > 64:
        raise ValueError("q: %d tokens; the layer takes at most 64, larger batches go %s"
                         % (T, "in pieces" if name == "moe_decode_layer_w4" else "through the masked GEMMs"))
    pq, ldq = _rows(q, "q", _E4M3, T, K)
    _typed(sf, "sf", _U32)
    if sf.dim() != 2 or sf.shape[0] != _words(K) or sf.shape[1] < T or sf.stride(1) != 1 or (
            sf.shape[0] > 1 and sf.stride(0) < T):
        raise ValueError("sf must be [%d, >= %d] with unit column stride, got shape %s strides %s"
                         % (_words(K), T, list(sf.shape), list(sf.stride())))
    pi = _whole(topk_ids, "topk_ids", _I32, (T, topk))
    pw = _whole(weights, "weights", _F32, (T, topk))
    wt, st = dtypes
    p = [_whole(w13, "w13", wt, shapes[0]), _whole(s13, "s13", st, shapes[1]), _whole(w2, "w2", wt, shapes[2]),
         _whole(s2, "s2", st, shapes[3])]
    pb, ld_b = (None, 0) if base is None else _rows(base, "base", _BF16, T, K)
    out, po, ld_o = _out_rows(out, "out", _BF16, T, K, q)
    # the gated activations of the pairs, from torch's allocator (the stream's, or a capture's own memory)
    need = _lib.moe_decode_layer_scratch_bytes(T, topk, H)
    scratch = q.new_empty(need, dtype=torch.uint8)
    _launch(name, (q, sf, topk_ids, weights, w13, s13, w2, s2, base), pq, ldq, sf.data_ptr(),
            sf.stride(0) if sf.shape[0] > 1 else max(T, 1), pi, pw, *p, pb, ld_b, T, topk, w13.shape[0], K, H, po, ld_o,
            scratch.data_ptr(), need)
    return out


def _moe_e4m3(name, q, sf, topk_ids, weights, w13, s13, w2, s2, base, out):
    if w13.dim() != 3 or w2.dim() != 3 or w13.shape[1] % 256 or w13.shape[2] % 128:
        raise ValueError("w13 must be [E, 2H, K] and w2 [E, K, H] with H and K multiples of 128")
    E, H, K = w13.shape[0], w13.shape[1] // 2, w13.shape[2]
    if q.dim() == 2 and q.shape[1] != K:
        raise ValueError("q and w13 disagree on K")
    shapes = (E, 2 * H, K), (E, H // 64, K // 128), (E, K, H), (E, K // 128, H // 128)
    return _moe(name, q, sf, topk_ids, weights, w13, s13, w2, s2, H, shapes, (_E4M3, _F32), base, out)


def moe_decode_layer(q: torch.Tensor, sf: torch.Tensor, topk_ids: torch.Tensor, weights: torch.Tensor,
                     w13: torch.Tensor, s13: torch.Tensor, w2: torch.Tensor, s2: torch.Tensor,
                     base: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """A mixture-of-experts layer for at most 64 tokens in two launches: gate_up product, SiLU, quantization, down
    product, and the weighted sum over each token's experts on top of base.  q uint8 [T, K] and sf int32
    [ceil(K/512), >= T] (as fp8_quant_group_pack or residual_rms_norm give them), topk_ids int32 and weights fp32
    [T, topk] (as moe_route_topk gives them; ids outside [0, E) are left out), w13 e4m3 [E, 2H, K] with fp32 block scales
    [E, 2H/128, K/128], w2 [E, K, H] with [E, K/128, H/128], base bf16 [T, K] -> bf16 [T, K]."""
    if stream is not None:
        return _on_stream(stream, moe_decode_layer, q, sf, topk_ids, weights, w13, s13, w2, s2, base, out)
    return _moe_e4m3("moe_decode_layer", q, sf, topk_ids, weights, w13, s13, w2, s2, base, out)


def moe_decode_layer_preshuffled(q: torch.Tensor, sf: torch.Tensor, topk_ids: torch.Tensor, weights: torch.Tensor,
                                 w13: torch.Tensor, s13: torch.Tensor, w2: torch.Tensor, s2: torch.Tensor,
                                 base: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                 stream=None) -> torch.Tensor:
    """moe_decode_layer on weights in the layout of fp8_weight_preshuffle (same shapes)."""
    if stream is not None:
        return _on_stream(stream, moe_decode_layer_preshuffled, q, sf, topk_ids, weights, w13, s13, w2, s2, base, out)
    return _moe_e4m3("moe_decode_layer_preshuffled", q, sf, topk_ids, weights, w13, s13, w2, s2, base, out)


def moe_decode_layer_w4(q: torch.Tensor, sf: torch.Tensor, topk_ids: torch.Tensor, weights: torch.Tensor,
                        w13: torch.Tensor, s13: torch.Tensor, w2: torch.Tensor, s2: torch.Tensor,
                        base: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """moe_decode_layer on e2m1 weights as w4_preshuffle lays them out: w13 uint8 [E, 2H/16, K/128, 1024] with s13
    uint8 [E, 2H/16, ceil(K/512), 64, 4], w2 [E, K/16, H/128, 1024] with s2 [E, K/16, ceil(H/512), 64, 4].
    The masked GEMMs take no such weights: more than 64 tokens go in pieces of 64, each of which reads its experts again."""
    if stream is not None:
        return _on_stream(stream, moe_decode_layer_w4, q, sf, topk_ids, weights, w13, s13, w2, s2, base, out)
    if w13.dim() != 4 or w2.dim() != 4 or w13.shape[1] % 16:
        raise ValueError("w13 must be [E, 2H/16, K/128, 1024] and w2 [E, K/16, H/128, 1024] with H a multiple of 128")
    E, H, K = w13.shape[0], 8 * w13.shape[1], 128 * w13.shape[2]
    if q.dim() == 2 and q.shape[1] != K:
        raise ValueError("q and w13 disagree on K")
    shapes = ((E, H // 8, K // 128, 1024), (E, H // 8, _words(K), 64, 4), (E, K // 16, H // 128, 1024),
              (E, K // 16, _words(H), 64, 4))
    return _moe("moe_decode_layer_w4", q, sf, topk_ids, weights, w13, s13, w2, s2, H, shapes, (_U8, _U8), base, out)


def _group(format, group):
    if format not in _FORMAT:
        raise ValueError("format must be 'int4' or 'e2m1', got %r" % (format,))
    if group is None:
        group = 32 if format == "e2m1" else 128
    if group not in ((32,) if format == "e2m1" else (32, 64, 128)):
        raise ValueError("group must be 32, or for int4 32, 64 or 128, got %r" % (group,))
    return group


def w4_group_quant(w: torch.Tensor, format: str = "int4", group: int | None = None, zero_points: bool = False,
                   codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                   zeros: torch.Tensor | None = None, stream=None):
    """Weights to 4 bits under group scales.  w bf16 [..., N, K] -> (codes uint8 [..., N, K/2], scales [..., N, K/group],
    zeros uint8 [..., N, K/group] or None).  format "int4": scales bf16, group 32, 64 or 128 (the default), with
    zero_points a zero point for each group; "e2m1": UE8M0 bytes as uint8, group 32."""
    if stream is not None:
        return _on_stream(stream, w4_group_quant, w, format, group, zero_points, codes, scales, zeros)
    group = _group(format, group)
    if w.dim() < 2 or w.shape[-1] % 128:
        raise ValueError("w must be [..., N, K] with K a multiple of 128, got %s" % list(w.shape))
    if format == "e2m1" and zero_points:
        raise ValueError("zero points are of int4 only")
    if zeros is not None and not zero_points:
        raise ValueError("zeros are written with zero_points only")
    K = w.shape[-1]
    pw = _whole(w, "w", _BF16, w.shape)
    codes, pc = _out(codes, "codes", _U8, (*w.shape[:-1], K // 2), w)
    scales, ps = _out(scales, "scales", _U8 if format == "e2m1" else _BF16, (*w.shape[:-1], K // group), w)
    pz = None
    if zero_points:
        zeros, pz = _out(zeros, "zeros", _U8, (*w.shape[:-1], K // group), w)
    _launch("w4_group_quant", (w,), pw, w.numel() // K if K else 0, K, _FORMAT[format], group, pc, ps, pz)
    return codes, scales, zeros


def _format_of(scales):
    if scales.dtype not in (torch.uint8, torch.bfloat16):
        raise TypeError("scales: dtype %s; uint8 (e2m1) or bfloat16 (int4)" % scales.dtype)
    return "e2m1" if scales.dtype == torch.uint8 else "int4"


def w4_preshuffle(codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None, stream=None):
    """Codes [N, K/2] or [E, N, K/2], scales (uint8: e2m1, bfloat16: int4) and zero points in row order -> the layout of
    w4_group_gemv_nt and moe_decode_layer_w4, tiles = ceil(N/16) and units = ceil(K/512): (codes [(E,) tiles, K/128,
    1024], scales [(E,) tiles, units, 64, 4] for e2m1 or [(E,) tiles, units, 16, 512/group], zeros like scales or None)."""
    if stream is not None:
        return _on_stream(stream, w4_preshuffle, codes, scales, zeros)
    if codes.dim() not in (2, 3) or codes.shape[-1] % 64 or codes.shape[-1] == 0:
        raise ValueError("codes must be [N, K/2] or [E, N, K/2] with K a multiple of 128, got %s" % list(codes.shape))
    *lead, N, half = codes.shape
    K = 2 * half
    format = _format_of(scales)
    if scales.dim() != codes.dim() or scales.shape[-1] < 1 or K % scales.shape[-1]:
        raise ValueError("scales must be [..., N, K/group], got %s" % list(scales.shape))
    group = _group(format, K // scales.shape[-1])
    if format == "e2m1" and zeros is not None:
        raise ValueError("zero points are of int4 only")
    pc = _whole(codes, "codes", _U8, codes.shape)
    ps = _whole(scales, "scales", (scales.dtype,), (*lead, N, K // group))
    pz = None if zeros is None else _whole(zeros, "zeros", _U8, (*lead, N, K // group))
    tiles, units = (N + 15) // 16, _words(K)
    shape = (*lead, tiles, units, *((64, 4) if format == "e2m1" else (16, 512 // group)))
    codes_out = codes.new_empty((*lead, tiles, K // 128, 1024))
    scales_out = scales.new_empty(shape)
    zeros_out = None if zeros is None else zeros.new_empty(shape)
    _launch("w4_preshuffle", (codes, scales, zeros), pc, ps, pz, lead[0] if lead else 1, N, K, _FORMAT[format], group,
            codes_out.data_ptr(), scales_out.data_ptr(), None if zeros is None else zeros_out.data_ptr())
    return codes_out, scales_out, zeros_out


def w4_group_gemv_nt(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, n: int,
                     zeros: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x bf16 [T, K] times the n rows of 4-bit weights that w4_preshuffle laid out: codes uint8 [ceil(n/16), K/128, 1024],
    scales uint8 [ceil(n/16), ceil(K/512), 64, 4] (e2m1) or bf16 [ceil(n/16), ceil(K/512), 16, 512/group] (int4), zeros
    uint8 like the scales or None -> bf16 [T, n].  Made for few tokens: every 64 of them read the weights once."""
    if stream is not None:
        return _on_stream(stream, w4_group_gemv_nt, x, codes, scales, n, zeros, out)
    T, K = _2d(x, "x")
    px, ldx = _rows(x, "x", _BF16, T, K)
    if K % 128 or K == 0:
        raise ValueError("K must be a multiple of 128, got %d" % K)
    n = operator.index(n)
    if n < 0:
        raise ValueError("n must not be negative, got %d" % n)
    tiles, units = (n + 15) // 16, _words(K)
    pc = _whole(codes, "codes", _U8, (tiles, K // 128, 1024))
    pz = None
    if scales.dtype == torch.uint8:
        format, group = 0, 32
        if zeros is not None:
            raise ValueError("zero points are of int4 only")
        ps = _whole(scales, "scales", _U8, (tiles, units, 64, 4))
    else:
        _typed(scales, "scales", _BF16)
        per = scales.shape[-1] if scales.dim() == 4 else 0
        if per not in (4, 8, 16):
            raise ValueError("scales must be [%d, %d, 16, 512/group], got %s" % (tiles, units, list(scales.shape)))
        format, group = 1, 512 // per
        ps = _whole(scales, "scales", _BF16, (tiles, units, 16, per))
        if zeros is not None:
            pz = _whole(zeros, "zeros", _U8, (tiles, units, 16, per))
    out, po, ld_o = _out_rows(out, "out", _BF16, T, n, x)
    _launch("w4_group_gemv_nt", (x, codes, scales, zeros), px, ldx, pc, ps, pz, T, n, K, format, group, po, ld_o)
    return out
