"""The operators around the experts' products refuse wrong arguments before anything is
launched: the binding by shape, type and stride (driven with host tensors: a call that passes those checks fails only at
"must be a device tensor"), the C ABI by status."""
import ctypes

import pytest
import torch

import block_scaled_fp8_token_amd as F
from block_scaled_fp8_token_amd import _lib

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN = 0, -1, -2, -3
A, B, C, D, S, I, W = (0x100000 * i for i in range(1, 8))  # 256-byte aligned, never dereferenced
bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def refuses(error, match, fn, *args, **kw):
    with pytest.raises(error, match=match):
        fn(*args, **kw)


def passes_checks(fn, *args, **kw):
    refuses(ValueError, "device tensor", fn, *args, **kw)


def test_route_binding():
    passes_checks(F.moe_route_topk, z(5, 60), 6)
    passes_checks(F.moe_route_topk, z(5, 80, dtype=f32)[:, :60], 6, bias=z(60, dtype=f32), scoring="sigmoid")
    refuses(TypeError, "logits", F.moe_route_topk, z(5, 60, dtype=torch.float16), 6)
    refuses(ValueError, "logits", F.moe_route_topk, z(60), 6)
    refuses(ValueError, "logits", F.moe_route_topk, z(60, 5).t(), 6)
    refuses(ValueError, "bias", F.moe_route_topk, z(5, 60), 6, bias=z(59, dtype=f32))
    refuses(TypeError, "bias", F.moe_route_topk, z(5, 60), 6, bias=z(60))
    refuses(ValueError, "scoring", F.moe_route_topk, z(5, 60), 6, scoring="tanh")
    refuses(ValueError, "topk_ids", F.moe_route_topk, z(5, 60), 6, topk_ids=z(5, 5, dtype=i32))
    refuses(TypeError, "topk_ids", F.moe_route_topk, z(5, 60), 6, topk_ids=z(5, 6, dtype=torch.int64))
    refuses(ValueError, "weights", F.moe_route_topk, z(5, 60), 6, weights=z(4, 6, dtype=f32))
    passes_checks(F.moe_route_topk_backward, z(5, 60), z(5, 6, dtype=i32), z(5, 6, dtype=f32))
    refuses(ValueError, "d_weights", F.moe_route_topk_backward, z(5, 60), z(5, 6, dtype=i32), z(5, 7, dtype=f32))
    refuses(ValueError, "topk_ids", F.moe_route_topk_backward, z(5, 60), z(4, 6, dtype=i32), z(5, 6, dtype=f32))
    refuses(TypeError, "d_logits", F.moe_route_topk_backward, z(5, 60), z(5, 6, dtype=i32), z(5, 6, dtype=f32),
            d_logits=z(5, 60, dtype=f32))


def test_combine_binding():
    y, ids, w = z(4, 16, 64), z(7, 2, dtype=i32), z(7, 2, dtype=f32)
    passes_checks(F.moe_combine, y, ids, ids, w, base=z(7, 64))
    refuses(ValueError, "y must", F.moe_combine, z(16, 64), ids, ids)
    refuses(ValueError, "y must be contiguous", F.moe_combine, z(16, 4, 64).transpose(0, 1), ids, ids)
    refuses(ValueError, "slot_of", F.moe_combine, y, ids, z(7, 3, dtype=i32))
    refuses(TypeError, "weights", F.moe_combine, y, ids, ids, z(7, 2))
    refuses(ValueError, "base", F.moe_combine, y, ids, ids, base=z(7, 72))
    refuses(ValueError, "base", F.moe_combine, y, ids, ids, base=z(64, 7).t())
    refuses(ValueError, "out", F.moe_combine, y, ids, ids, out=z(6, 64))
    d = z(7, 64)
    passes_checks(F.moe_combine_backward, d, y, ids, ids, w)
    passes_checks(F.moe_combine_backward, z(7, 128), z(4, 16, 128), ids, ids, quantize=True)
    refuses(ValueError, "d_out", F.moe_combine_backward, z(7, 56), y, ids, ids, w)
    refuses(ValueError, "without weights", F.moe_combine_backward, d, y, ids, ids, d_weights=w)
    refuses(ValueError, "d_y", F.moe_combine_backward, d, y, ids, ids, w, d_y=z(4, 15, 64))
    refuses(ValueError, "quantize", F.moe_combine_backward, d, y, ids, ids, w, quantize=True, d_y=y)
    refuses(ValueError, "quantize", F.moe_combine_backward, d, y, ids, ids, w, q=z(4, 16, 64, dtype=u8))
    refuses(ValueError, "sf", F.moe_combine_backward, z(7, 128), z(4, 16, 128), ids, ids, quantize=True,
            sf=z(4, 2, 16, dtype=i32))


def test_norm_binding():
    x, w = z(5, 128), z(128)
    passes_checks(F.residual_rms_norm, x, w)
    passes_checks(F.residual_rms_norm, x.float(), w, y=x, w_post=w, gate=z(5, 128), out="both")
    refuses(ValueError, "x must", F.residual_rms_norm, z(128), w)
    refuses(ValueError, "w_pre", F.residual_rms_norm, x, z(64))
    refuses(TypeError, "w_pre", F.residual_rms_norm, x, w.float())
    refuses(ValueError, "apply to y", F.residual_rms_norm, x, w, w_post=w)
    refuses(ValueError, "apply to y", F.residual_rms_norm, x, w, gate=w)
    refuses(ValueError, "y must", F.residual_rms_norm, x, w, y=z(4, 128))
    refuses(ValueError, "gate", F.residual_rms_norm, x, w, y=x, gate=z(4, 128))
    refuses(ValueError, "out must", F.residual_rms_norm, x, w, out="e5m2")
    refuses(TypeError, "h:", F.residual_rms_norm, x, w, y=x, h=x.float())
    refuses(ValueError, "z is not", F.residual_rms_norm, x, w, out="fp8", z=x)
    refuses(ValueError, "are not written", F.residual_rms_norm, x, w, q=z(5, 128, dtype=u8))
    refuses(ValueError, "sf must", F.residual_rms_norm, x, w, out="fp8", sf=z(1, 4, dtype=i32))
    passes_checks(F.residual_rms_norm_backward, x, x, w)
    passes_checks(F.residual_rms_norm_backward, x, x.float(), w, d_h=x.float(), y=x, w_post=w, gate=w)
    refuses(ValueError, "d_z", F.residual_rms_norm_backward, z(4, 128), x, w)
    refuses(TypeError, "d_h", F.residual_rms_norm_backward, x, x, w, d_h=x.float())
    refuses(ValueError, "apply to y", F.residual_rms_norm_backward, x, x, w, gate=w)
    refuses(ValueError, "not there", F.residual_rms_norm_backward, x, x, w, y=x, d_w_post=w.float())
    refuses(TypeError, "d_gate", F.residual_rms_norm_backward, x, x, w, y=x, gate=w, d_gate=w)


def test_checkpoint_binding():
    x, m = z(3, 8, 512), z(3, dtype=i32)
    passes_checks(F.silu_mul_quant_group_pack_checkpoint, x, m)
    refuses(ValueError, "x must", F.silu_mul_quant_group_pack_checkpoint, z(8, 512), m)
    refuses(ValueError, "masked_m", F.silu_mul_quant_group_pack_checkpoint, x, z(4, dtype=i32))
    refuses(ValueError, "cq", F.silu_mul_quant_group_pack_checkpoint, x, m, cq=z(3, 8, 256, dtype=u8))
    refuses(ValueError, "csf", F.silu_mul_quant_group_pack_checkpoint, x, m, csf=z(3, 1, 8, dtype=i32))
    d, cq, csf = z(3, 8, 256), z(3, 8, 512, dtype=u8), z(3, 2, 8, dtype=i32)
    passes_checks(F.silu_mul_backward_from_checkpoint, d, m, cq, csf)
    passes_checks(F.silu_mul_backward_from_checkpoint, d, m, cq, csf, quantize=True)
    refuses(ValueError, "csf", F.silu_mul_backward_from_checkpoint, d, m, cq, z(3, 1, 8, dtype=i32))
    refuses(ValueError, "d_x", F.silu_mul_backward_from_checkpoint, d, m, cq, csf, d_x=z(3, 8, 256))
    refuses(ValueError, "quantize", F.silu_mul_backward_from_checkpoint, d, m, cq, csf, quantize=True, d_x=z(3, 8, 512))
    refuses(ValueError, "quantize", F.silu_mul_backward_from_checkpoint, d, m, cq, csf, q=cq)


def _route(logits=A, f32=0, ld=256, T=4, E=256, bias=None, scoring=0, groups=1, topk_groups=1, group_top=1, topk=8,
           ids=I, weights=W):
    return _lib.moe_route_topk(logits, f32, ld, T, E, bias, scoring, groups, topk_groups, group_top, topk, 1, 1.0, ids,
                               weights, None)


@pytest.mark.parametrize("bad", [dict(E=0), dict(E=1025, ld=1025), dict(ld=255), dict(T=-1), dict(topk=0), dict(topk=65),
                                 dict(topk=257), dict(groups=3), dict(groups=0), dict(groups=128), dict(topk_groups=2),
                                 dict(topk_groups=0), dict(groups=64, topk_groups=1), dict(group_top=3), dict(group_top=0),
                                 dict(E=4, topk=2, group_top=2, groups=4, topk_groups=4), dict(scoring=2), dict(f32=2)])
def test_route_status_shape(bad):
    assert _route(**bad) == ERR_SHAPE


def test_route_status():
    assert _route(T=0, logits=None, ids=None, weights=None) == OK
    assert _route(logits=None) == ERR_NULL and _route(ids=None) == ERR_NULL and _route(weights=None) == ERR_NULL
    assert _route(logits=A + 1) == ERR_ALIGN and _route(logits=A + 2, f32=1) == ERR_ALIGN
    assert _route(bias=B + 2) == ERR_ALIGN and _route(ids=I + 1) == ERR_ALIGN

    def back(logits=A, ld=256, T=4, E=256, ids=I, dw=W, topk=8, d=D, ld_d=256):
        return _lib.moe_route_topk_backward(logits, 0, ld, T, E, ids, dw, 0, topk, 1, 1.0, d, ld_d, None)
    assert back(ld_d=255) == ERR_SHAPE and back(topk=65) == ERR_SHAPE and back(d=None) == ERR_NULL
    assert back(dw=None) == ERR_NULL and back(d=D + 1) == ERR_ALIGN and back(T=0) == OK


def test_combine_status():
    def fwd(y=A, ids=I, slots=S, w=W, base=None, ld_base=0, T=4, topk=2, E=3, M=16, N=64, out=C, ld_out=64):
        return _lib.moe_combine(y, ids, slots, w, base, ld_base, T, topk, E, M, N, out, ld_out, None)
    assert fwd(N=60) == ERR_SHAPE and fwd(topk=0) == ERR_SHAPE and fwd(topk=65) == ERR_SHAPE and fwd(T=-1) == ERR_SHAPE
    assert fwd(ld_out=56) == ERR_SHAPE and fwd(base=B, ld_base=56) == ERR_SHAPE and fwd(E=-1) == ERR_SHAPE
    assert fwd(T=1 << 33) == ERR_SHAPE and fwd(T=(1 << 22) + 1) == ERR_SHAPE and fwd(N=1 << 21, ld_out=1 << 21) == ERR_SHAPE
    assert _route(T=(1 << 22) + 1) == ERR_SHAPE
    assert fwd(y=None) == ERR_NULL and fwd(out=None) == ERR_NULL and fwd(slots=None) == ERR_NULL
    assert fwd(y=A + 8) == ERR_ALIGN and fwd(ld_out=68) == ERR_ALIGN and fwd(base=B, ld_base=68) == ERR_ALIGN
    assert fwd(T=0, y=None) == OK and fwd(N=0) == OK

    def back(d=A, ld=128, y=B, ids=I, slots=S, w=W, T=4, topk=2, E=3, M=16, N=128, dy=C, q=None, sf=None, dw=D):
        return _lib.moe_combine_backward(d, ld, y, ids, slots, w, T, topk, E, M, N, dy, q, sf, dw, None)
    assert back(dy=None) == ERR_NULL and back(q=C, sf=S) == ERR_NULL      # neither, or both
    assert back(dy=None, q=C) == ERR_NULL and back(y=None) == ERR_NULL and back(d=None) == ERR_NULL
    assert back(dy=None, q=C, sf=S, N=64) == ERR_SHAPE and back(ld=120) == ERR_SHAPE
    assert back(dy=C + 8) == ERR_ALIGN and back(ld=132) == ERR_ALIGN and back(dw=D + 2) == ERR_ALIGN
    assert back(T=0) == OK


def _norm(x=A, ldx=128, f32=0, y=B, ldy=128, w_post=W, gate=None, ld_gate=0, w_pre=W, T=4, N=128, h=C, ldh=128, z=D,
          ldz=128, q=None, ldq=0, sf=None, ld_sf=0):
    return _lib.residual_rms_norm(x, ldx, f32, y, ldy, w_post, gate, ld_gate, w_pre, 1.0, 1e-6, 0.0, T, N, h, ldh, z, ldz,
                                  q, ldq, sf, ld_sf, None)


def test_norm_status():
    assert _norm(N=124) == ERR_SHAPE and _norm(N=16392, ldx=16392) == ERR_SHAPE and _norm(T=-1) == ERR_SHAPE
    assert _norm(ldx=120) == ERR_SHAPE and _norm(ldy=120) == ERR_SHAPE and _norm(ldh=120) == ERR_SHAPE
    assert _norm(q=S, ldq=128, sf=I, ld_sf=3) == ERR_SHAPE and _norm(gate=S, ld_gate=120) == ERR_SHAPE
    assert _norm(N=120, q=S, ldq=128, sf=I, ld_sf=4) == ERR_SHAPE and _norm(f32=2) == ERR_SHAPE
    assert _norm(x=None) == ERR_NULL and _norm(w_pre=None) == ERR_NULL and _norm(h=None, z=None) == ERR_NULL
    assert _norm(y=None) == ERR_NULL and _norm(y=None, w_post=None, gate=S) == ERR_NULL  # w_post, gate without y
    assert _norm(q=S, ldq=128) == ERR_NULL and _norm(sf=S, ld_sf=4) == ERR_NULL
    assert _norm(x=A + 8) == ERR_ALIGN and _norm(ldx=132) == ERR_ALIGN and _norm(w_post=W + 2) == ERR_ALIGN
    assert _norm(q=S, ldq=136, sf=I, ld_sf=4) == ERR_ALIGN and _norm(gate=S, ld_gate=132) == ERR_ALIGN
    assert _norm(T=0, x=None, y=None, h=None, z=None) == OK and _norm(N=0) == OK

    def back(dz=A, dh=None, h=B, y=C, w_post=W, gate=None, ld_gate=0, w_pre=W, T=4, N=128, dx=D, dy=S, dwp=I, dwo=I,
             dg=None, ld_dg=0):
        return _lib.residual_rms_norm_backward(dz, 128, dh, 128, h, 128, 0, y, 128, w_post, gate, ld_gate, w_pre, 1.0,
                                               1e-6, 0.0, T, N, dx, 128, dy, 128, dwp, dwo, dg, ld_dg, None)
    assert back(dz=None) == ERR_NULL and back(dx=None) == ERR_NULL and back(dwp=None) == ERR_NULL
    assert back(dy=None) == ERR_NULL and back(dwo=None) == ERR_NULL and back(gate=S) == ERR_NULL and back(dg=S) == ERR_NULL
    assert back(N=136) == ERR_SHAPE and back(gate=S, ld_gate=128, dg=S, ld_dg=120) == ERR_SHAPE
    assert back(dwp=I + 4) == ERR_ALIGN and back(dh=A + 2) == ERR_ALIGN
    assert back(gate=S, ld_gate=128, dg=S, ld_dg=132) == ERR_ALIGN


def test_checkpoint_status():
    def fwd(x=A, m=I, E=3, M=8, H=256, q=B, sf=S, cq=C, csf=W):
        return _lib.silu_mul_quant_group_pack_checkpoint(x, m, E, M, H, q, sf, cq, csf, None)
    assert fwd(H=200) == ERR_SHAPE and fwd(E=1025) == ERR_SHAPE and fwd(M=-1) == ERR_SHAPE
    assert fwd(cq=None) == ERR_NULL and fwd(m=None) == ERR_NULL and fwd(x=A + 8) == ERR_ALIGN and fwd(csf=W + 2) == ERR_ALIGN
    assert fwd(E=0) == OK and fwd(M=0) == OK and fwd(H=0) == OK

    def back(d=A, m=I, E=3, M=8, H=256, cq=B, csf=S, dx=C, q=None, sf=None):
        return _lib.silu_mul_backward_from_checkpoint(d, m, E, M, H, cq, csf, dx, q, sf, None)
    assert back(dx=None) == ERR_NULL and back(q=D, sf=W) == ERR_NULL and back(dx=None, q=D) == ERR_NULL
    assert back(H=64) == ERR_SHAPE and back(d=A + 4) == ERR_ALIGN and back(E=0) == OK


def test_signatures_match_the_header():
    # every argument of the new entry points is typed (ctypes would otherwise pass 32-bit integers)
    for n in F.block_ops.__all__:
        assert getattr(_lib, n).argtypes and getattr(_lib, n).restype is ctypes.c_int
