"""The operators of a decode step refuse wrong arguments before anything is launched: the binding by
shape, type and stride (driven with host tensors: a call that passes those checks fails only at "must be
a device tensor"), the C ABI by status."""
import pytest
import torch

import block_scaled_fp8_token_amd as F
import decode_reference as R
from block_scaled_fp8_token_amd import _lib

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_SCRATCH = 0, -1, -2, -3, -7
Q, SF, I, W, W13, S13, W2, S2, BASE, OUT, SCRATCH = (0x100000 * i for i in range(1, 12))  # never dereferenced
bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def refuses(error, match, fn, *args, **kw):
    with pytest.raises(error, match=match):
        fn(*args, **kw)


def passes_checks(fn, *args, **kw):
    refuses(ValueError, "device tensor", fn, *args, **kw)


E, K, H, T, TOPK = 3, 640, 256, 5, 2


def layer_args(kind):
    a = dict(q=z(T, K, dtype=u8), sf=z(2, 8, dtype=i32), topk_ids=z(T, TOPK, dtype=i32), weights=z(T, TOPK, dtype=f32))
    if kind == "w4":
        a.update(w13=z(E, 2 * H // 16, K // 128, 1024, dtype=u8), s13=z(E, 2 * H // 16, 2, 64, 4, dtype=u8),
                 w2=z(E, K // 16, H // 128, 1024, dtype=u8), s2=z(E, K // 16, 1, 64, 4, dtype=u8))
    else:
        a.update(w13=z(E, 2 * H, K, dtype=u8), s13=z(E, 2 * H // 128, K // 128, dtype=f32), w2=z(E, K, H, dtype=u8),
                 s2=z(E, K // 128, H // 128, dtype=f32))
    return a


CALLS = {"plain": F.moe_decode_layer, "preshuffled": F.moe_decode_layer_preshuffled, "w4": F.moe_decode_layer_w4}


@pytest.mark.parametrize("kind", list(CALLS))
def test_layer_binding(kind):
    fn, good = CALLS[kind], layer_args(kind)

    def bad(error, match, **kw):
        refuses(error, match, fn, **{**good, **kw})
    passes_checks(fn, **good)
    passes_checks(fn, **{**good, "base": z(T, K + 8)[:, :K], "out": z(T, K)})
    passes_checks(fn, **{**good, "q": z(T, K + 16, dtype=u8)[:, :K]})
    if kind != "w4":
        passes_checks(fn, **{**good, "w13": good["w13"].view(torch.float8_e4m3fn), "w2": good["w2"].view(torch.float8_e4m3fn)})
    bad(ValueError, "q must have 2", q=z(K, dtype=u8))
    bad(TypeError, "q", q=z(T, K))
    bad(ValueError, "disagree", q=z(T, 512, dtype=u8))
    bad(ValueError, "q must", q=z(K, T, dtype=u8).t())
    bad(ValueError, "at most 64", q=z(65, K, dtype=u8))
    bad(TypeError, "sf", sf=z(2, 8, dtype=f32))
    bad(ValueError, "sf must", sf=z(1, 8, dtype=i32))
    bad(ValueError, "sf must", sf=z(2, 4, dtype=i32))
    bad(ValueError, "sf must", sf=z(8, 2, dtype=i32).t())
    bad(ValueError, "topk_ids", topk_ids=z(T + 1, TOPK, dtype=i32))
    bad(TypeError, "topk_ids", topk_ids=z(T, TOPK, dtype=torch.int64))
    bad(ValueError, "weights", weights=z(T, TOPK + 1, dtype=f32))
    bad(TypeError, "weights", weights=z(T, TOPK))
    bad(TypeError, "w13", w13=good["w13"].float())
    bad(ValueError, "w13", w13=good["w13"][:, :-1])
    bad(ValueError, "w13", w13=good["w13"][0])
    bad(ValueError, "w2", w2=good["w2"][:, :-1])
    bad(ValueError, "w2", w2=good["w2"][:2])
    bad(ValueError, "s13", s13=good["s13"][:, :-1])
    bad(ValueError, "s2", s2=good["s2"][:2])
    bad(TypeError, "s2", s2=good["s2"].to(torch.float64))
    bad(ValueError, "w2 must be contiguous", w2=good["w2"].transpose(0, 1).contiguous().transpose(0, 1))
    bad(ValueError, "base", base=z(T, K + 1))
    bad(TypeError, "base", base=z(T, K, dtype=f32))
    bad(ValueError, "device", out=z(T, K, dtype=bf).to("meta"))


@pytest.mark.parametrize("kind,way", [("plain", "masked GEMMs"), ("preshuffled", "masked GEMMs"), ("w4", "in pieces")])
def test_layer_names_a_way_for_larger_batches(kind, way):
    """One that exists: the masked GEMMs take no e2m1 weights."""
    with pytest.raises(ValueError, match=way) as refusal:
        CALLS[kind](**{**layer_args(kind), "q": z(65, K, dtype=u8)})
    assert ("masked" in str(refusal.value)) == (kind != "w4")


def test_w4_binding():
    passes_checks(F.w4_group_quant, z(5, 256))
    passes_checks(F.w4_group_quant, z(2, 5, 256), "int4", 32, True)
    passes_checks(F.w4_group_quant, z(5, 256), "e2m1")
    refuses(ValueError, "format", F.w4_group_quant, z(5, 256), "fp4")
    refuses(ValueError, "group", F.w4_group_quant, z(5, 256), "int4", 16)
    refuses(ValueError, "group", F.w4_group_quant, z(5, 256), "e2m1", 64)
    refuses(ValueError, "zero points", F.w4_group_quant, z(5, 256), "e2m1", zero_points=True)
    refuses(ValueError, "zeros are written", F.w4_group_quant, z(5, 256), zeros=z(5, 2, dtype=u8))
    refuses(ValueError, "multiple of 128", F.w4_group_quant, z(5, 200))
    refuses(ValueError, "w must", F.w4_group_quant, z(256))
    refuses(ValueError, "contiguous", F.w4_group_quant, z(256, 128).t())
    refuses(TypeError, "w:", F.w4_group_quant, z(5, 256, dtype=f32))
    refuses(ValueError, "codes", F.w4_group_quant, z(5, 256), codes=z(5, 256, dtype=u8))
    c, s = z(20, 128, dtype=u8), z(20, 4)
    passes_checks(F.w4_preshuffle, c, s)
    passes_checks(F.w4_preshuffle, c, s, z(20, 4, dtype=u8))
    passes_checks(F.w4_preshuffle, c, z(20, 8, dtype=u8))
    passes_checks(F.w4_preshuffle, z(3, 20, 128, dtype=u8), z(3, 20, 2))
    refuses(ValueError, "codes must", F.w4_preshuffle, z(20, 100, dtype=u8), s)
    refuses(ValueError, "codes must", F.w4_preshuffle, z(128, dtype=u8), s)
    refuses(TypeError, "scales", F.w4_preshuffle, c, z(20, 4, dtype=f32))
    refuses(ValueError, "scales", F.w4_preshuffle, c, z(19, 4))
    refuses(ValueError, "group", F.w4_preshuffle, c, z(20, 16))
    refuses(ValueError, "group", F.w4_preshuffle, c, z(20, 4, dtype=u8))
    refuses(ValueError, "scales", F.w4_preshuffle, c, z(20, 3))
    refuses(ValueError, "zero points", F.w4_preshuffle, c, z(20, 8, dtype=u8), z(20, 8, dtype=u8))
    refuses(ValueError, "zeros", F.w4_preshuffle, c, s, z(20, 8, dtype=u8))
    x, codes = z(3, 640), z(2, 5, 1024, dtype=u8)
    passes_checks(F.w4_group_gemv_nt, x, codes, z(2, 2, 64, 4, dtype=u8), 20)
    for per in (4, 8, 16):
        passes_checks(F.w4_group_gemv_nt, x, codes, z(2, 2, 16, per), 20, zeros=z(2, 2, 16, per, dtype=u8))
    refuses(ValueError, "codes", F.w4_group_gemv_nt, x, codes, z(2, 2, 16, 4), 40)
    refuses(ValueError, "codes", F.w4_group_gemv_nt, x[:, :512], codes, z(2, 2, 16, 4), 20)
    refuses(ValueError, "scales", F.w4_group_gemv_nt, x, codes, z(2, 1, 16, 4), 20)
    refuses(ValueError, "scales", F.w4_group_gemv_nt, x, codes, z(2, 2, 16, 5), 20)
    refuses(ValueError, "scales", F.w4_group_gemv_nt, x, codes, z(2, 2, 16, 4, dtype=u8), 20)
    refuses(TypeError, "scales", F.w4_group_gemv_nt, x, codes, z(2, 2, 16, 4, dtype=f32), 20)
    refuses(ValueError, "zero points", F.w4_group_gemv_nt, x, codes, z(2, 2, 64, 4, dtype=u8), 20,
            zeros=z(2, 2, 64, 4, dtype=u8))
    refuses(ValueError, "zeros", F.w4_group_gemv_nt, x, codes, z(2, 2, 16, 4), 20, zeros=z(2, 2, 16, 8, dtype=u8))
    refuses(ValueError, "K must", F.w4_group_gemv_nt, z(3, 600), codes, z(2, 2, 16, 4), 20)
    refuses(TypeError, "x:", F.w4_group_gemv_nt, x.float(), codes, z(2, 2, 16, 4), 20)
    refuses(ValueError, "x must", F.w4_group_gemv_nt, z(640, 3).t(), codes, z(2, 2, 16, 4), 20)
    refuses(ValueError, "n must", F.w4_group_gemv_nt, x, codes[:0], z(0, 2, 16, 4), -5)
    refuses(TypeError, "integer", F.w4_group_gemv_nt, x, codes, z(2, 2, 16, 4), 20.5)


def _layer(name, q=Q, ldq=640, sf=SF, ld_sf=8, ids=I, w=W, w13=W13, s13=S13, w2=W2, s2=S2, base=BASE, ld_base=640, T=5,
           topk=2, E=3, K=640, H=256, out=OUT, ld_out=640, scratch=SCRATCH, nbytes=1 << 20):
    return getattr(_lib, name)(q, ldq, sf, ld_sf, ids, w, w13, s13, w2, s2, base, ld_base, T, topk, E, K, H, out, ld_out,
                               scratch, nbytes, None)


@pytest.mark.parametrize("name", ["moe_decode_layer", "moe_decode_layer_preshuffled", "moe_decode_layer_w4"])
def test_layer_abi(name):
    def call(**kw):
        return _layer(name, **kw)
    for kw in (dict(T=-1), dict(T=65), dict(topk=0), dict(topk=65), dict(E=0), dict(E=1025), dict(K=0), dict(K=600),
               dict(K=65664, ldq=65664), dict(H=0), dict(H=200), dict(H=65664), dict(ldq=512), dict(ld_sf=4), dict(ld_base=512),
               dict(ld_out=512), dict(ldq=1 << 30), dict(ldq=1 << 40), dict(ld_sf=1 << 30), dict(ld_sf=1 << 62)):
        assert call(**kw) == ERR_SHAPE, kw
    for p in ("q", "sf", "ids", "w", "w13", "s13", "w2", "s2", "out", "scratch"):
        assert call(**{p: None}) == ERR_NULL, p
    for kw in (dict(q=Q + 8), dict(ldq=648), dict(sf=SF + 2), dict(ids=I + 1), dict(w=W + 2), dict(w13=W13 + 8),
               dict(s13=S13 + 2), dict(w2=W2 + 4), dict(s2=S2 + 2), dict(base=BASE + 8), dict(ld_base=644), dict(out=OUT + 2),
               dict(ld_out=644), dict(scratch=SCRATCH + 8)):
        assert call(**kw) == ERR_ALIGN, kw
    if name.endswith("w4"):
        assert call(s13=S13 + 4) == ERR_ALIGN and call(s2=S2 + 8) == ERR_ALIGN
    need = _lib.moe_decode_layer_scratch_bytes(5, 2, 256)
    assert call(nbytes=need - 1) == ERR_SCRATCH
    assert call(T=0, q=None, out=None, scratch=None) == OK


def test_scratch_bytes():
    f = _lib.moe_decode_layer_scratch_bytes
    assert f(0, 2, 256) == f(65, 2, 256) == f(1, 0, 256) == f(1, 65, 256) == f(1, 1, 0) == f(1, 1, 65664) == 0
    for T in (1, 8, 16, 17, 64):
        for topk in (1, 8, 64):
            for H in (128, 640, 2048, 65536):
                pairs = T * topk
                least = pairs * (H + 4 * -(-H // 512))  # codes and packed scale bytes
                assert f(T, topk, H) >= (max(least, 4 * pairs * H) if pairs <= 64 else least)


def test_w4_abi():
    q = _lib.w4_group_quant
    assert q(Q, -1, 256, 1, 128, W, SF, None, None) == ERR_SHAPE
    assert q(Q, 4, 200, 1, 128, W, SF, None, None) == ERR_SHAPE
    assert q(Q, 4, 256, 2, 128, W, SF, None, None) == ERR_SHAPE
    assert q(Q, 4, 256, 1, 16, W, SF, None, None) == ERR_SHAPE
    assert q(Q, 4, 256, 0, 64, W, SF, None, None) == ERR_SHAPE
    assert q(Q, 4, 256, 0, 32, W, SF, I, None) == ERR_SHAPE  # e2m1 has no zero points
    assert q(None, 4, 256, 1, 128, W, SF, None, None) == ERR_NULL
    assert q(Q + 8, 4, 256, 1, 128, W, SF, None, None) == ERR_ALIGN
    assert q(Q, 4, 256, 1, 128, W + 4, SF, None, None) == ERR_ALIGN
    assert q(None, 0, 256, 1, 128, None, None, None, None) == OK
    s = _lib.w4_preshuffle
    assert s(Q, SF, None, -1, 32, 256, 1, 128, W, S13, None, None) == ERR_SHAPE
    assert s(Q, SF, None, 1, 1 << 28, 256, 1, 128, W, S13, None, None) == ERR_SHAPE
    assert s(Q, SF, I, 1, 32, 256, 1, 128, W, S13, None, None) == ERR_NULL
    assert s(Q, SF, None, 1, 32, 256, 1, 128, W, S13, I, None) == ERR_NULL
    assert s(Q, SF, None, 1, 32, 256, 1, 128, W + 8, S13, None, None) == ERR_ALIGN
    assert s(Q, SF, None, 1, 32, 256, 1, 128, W, S13 + 8, None, None) == ERR_ALIGN
    assert s(None, None, None, 0, 32, 256, 1, 128, None, None, None, None) == OK
    g = _lib.w4_group_gemv_nt

    def call(x=Q, ldx=256, codes=W, scales=SF, zeros=None, T=5, N=20, K=256, format=1, group=128, out=OUT, ld_out=20):
        return g(x, ldx, codes, scales, zeros, T, N, K, format, group, out, ld_out, None)
    for kw in (dict(T=-1), dict(T=(1 << 21) + 1), dict(N=-1), dict(N=(1 << 27) + 1), dict(K=0), dict(K=200), dict(K=65664),
               dict(ldx=128), dict(ldx=1 << 28), dict(ldx=1 << 60), dict(ld_out=19), dict(format=3), dict(group=256),
               dict(format=0, group=32, zeros=I)):
        assert call(**kw) == ERR_SHAPE, kw
    for p in ("x", "codes", "scales", "out"):
        assert call(**{p: None}) == ERR_NULL, p
    for kw in (dict(x=Q + 8), dict(ldx=260), dict(codes=W + 8), dict(scales=SF + 8), dict(zeros=I + 8), dict(out=OUT + 1)):
        assert call(**kw) == ERR_ALIGN, kw
    assert call(T=0, x=None) == OK and call(N=0, x=None) == OK


def test_reference_pins():
    """The references themselves, against torch and by hand."""
    import numpy as np
    rng = np.random.default_rng(0)
    v = rng.standard_normal((4, 256)) * np.exp2(rng.integers(-6, 6, (4, 256)))
    q, off = R.quant_group(v, np.zeros_like(v))
    most = np.abs(v).reshape(4, 2, 128).max(-1)
    s = np.exp2(np.ceil(np.log2(most / 448)))
    ref = (torch.from_numpy(v.reshape(4, 2, 128) / s[..., None]).float().to(torch.float8_e4m3fn).double().numpy() * s[..., None])
    assert np.array_equal(q, ref.reshape(4, 256)) and not off.any()
    # a value in the middle between two codes, and one next to it
    w = np.zeros((1, 128))
    w[0, :3] = [448.0, 17.0, 17.0 + 1e-9]
    q, off = R.quant_group(w, np.full_like(w, 1e-6))
    assert q[0, 1] == 16 and q[0, 2] == 18 and off[0, 1] == off[0, 2] == 2 and off[0, 3] == 0
    # a largest magnitude at the border of two scales: under the larger one 0.01 is another multiple of the smallest step
    w[0, :3] = [448.0, 1.0, 0.01]
    q, off = R.quant_group(w, np.full_like(w, 1e-9))
    assert q[0, 2] == 5 * 2.0 ** -9 and abs(off[0, 2] - 2.0 ** -9) < 1e-12 and off[0, 1] == 0
    codes = np.array([[0x21, 0xF8] + [0] * 62], np.uint8)  # nibbles 1, 2, 8, 15
    assert R.w4_values(codes, np.full((1, 4), 128, np.uint8))[0, :4].tolist() == [1.0, 2.0, 0.0, -12.0]
    assert R.w4_values(codes, np.full((1, 1), 0.5))[0, :4].tolist() == [-3.5, -3.0, 0.0, 3.5]
    assert R.w4_values(codes, np.full((1, 1), 0.5), np.full((1, 1), 15, np.uint8))[0, :4].tolist() == [-7.0, -6.5, -3.5, 0.0]
    x = rng.standard_normal((3, 128))
    w13, w2 = rng.standard_normal((2, 256, 128)) / 12, rng.standard_normal((2, 128, 128)) / 12
    ids, weights = np.array([[0, 1], [1, -1], [1, 1]]), rng.random((3, 2))
    out, bound = R.moe_layer(x, ids, weights, w13, w2)
    for t in range(3):
        want = np.zeros(128)
        for j in range(2):
            if ids[t, j] >= 0:
                h = torch.from_numpy(w13[ids[t, j]] @ x[t])
                y = (torch.nn.functional.silu(h[:128]) * h[128:]).numpy()
                want += weights[t, j] * (w2[ids[t, j]] @ R.quant_group(y[None], 0 * y[None])[0][0])
        assert np.allclose(out[t], want, rtol=1e-12, atol=1e-12)
    assert (bound > 0).all() and np.median(bound) < 0.05
