"""The operators of a decode step on the GPU against references in 64 bits: 4-bit weights bit for
bit, products and layers within the rounding of their sums."""
import numpy as np
import pytest
import torch

import decode_reference as R

pytestmark = pytest.mark.gpu
F = pytest.importorskip("block_scaled_fp8_token_amd")
DEV = "cuda:0"


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a).to(DEV)


def bf16(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16)


def poisoned(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


# ---------------------------------------------------------------- 4-bit weights

@pytest.mark.parametrize("group,zero_points", [(32, False), (64, True), (128, False), (32, True), (128, True)])
def test_quant_int4(group, zero_points):
    rng = np.random.default_rng(group + zero_points)
    w = bf16(rng, 37, 640, std=0.05)
    w[3] = 0
    w[4, :128] = 0
    w[5] = w[5].abs()
    w[6] = -w[6].abs()
    w[7, 11] = 300.0
    w[8] *= 1e-38
    codes, scales, zeros = F.w4_group_quant(w.to(DEV), "int4", group, zero_points)
    c, s, z = R.quant_int4(w.float().numpy(), group, zero_points)
    assert torch.equal(scales.cpu().view(torch.int16), s.view(torch.int16))
    assert np.array_equal(R.nibbles(codes.cpu().numpy()), c)
    assert (zeros is None) == (not zero_points)
    if zero_points:
        assert np.array_equal(zeros.cpu().numpy(), z)


@pytest.mark.parametrize("group", [32, 128])
def test_quant_of_the_largest_values(group):
    """A group whose span is past fp32's range: s = bf16(span / 15) with the span in 64 bits."""
    w = torch.linspace(-1, 1, 128).repeat(3, 1).bfloat16()
    w[:, ::16], w[:, 15::16] = -1, 1
    w *= torch.finfo(torch.bfloat16).max
    codes, scales, zeros = F.w4_group_quant(w.to(DEV), "int4", group, True)
    s = torch.tensor(2 * torch.finfo(torch.bfloat16).max / 15, dtype=torch.float64).float().bfloat16().item()
    assert (scales.cpu().float() == s).all()
    zero = round(torch.finfo(torch.bfloat16).max / s)
    assert (zeros.cpu() == zero).all()
    want = (w.double() / s).round().add(zero).clamp(0, 15)
    # w / s is rounded to fp32 (by at most 8 * 2^-24) before its rounding to an integer, which matters next to a middle
    # alone: every value is on one, which is exact in fp32, or away from it
    off = ((w.double() / s) % 1 - 0.5).abs()
    assert ((off == 0) | (off > 2.0 ** -20)).all()
    assert np.array_equal(R.nibbles(codes.cpu().numpy()), want.numpy())


def test_quant_e2m1():
    rng = np.random.default_rng(1)
    w = bf16(rng, 2, 40, 384, std=0.05)
    w[0, 0] = 0
    w[0, 1, :32] = torch.tensor(R.E2M1[np.arange(32) % 16], dtype=torch.bfloat16) * 0.25
    # every middle between two codes, with 6 among them so that the scale is 1
    mids = (R.E2M1[:7] + R.E2M1[1:8]) / 2
    w[0, 2, :32] = torch.tensor(np.resize(np.concatenate([mids, -mids, [6.0, -0.0]]), 32), dtype=torch.bfloat16)
    w[0, 3] *= 2.0 ** -120
    w[0, 4] *= 2.0 ** 100
    for i, m in enumerate((5.96875, 6.0, 6.03125, 12.0, 12.0625)):  # largest magnitudes around a power's border
        w[1, i] = w[1, i].clamp(-1, 1)
        w[1, i, 5::32] = m
    codes, scales, zeros = F.w4_group_quant(w.to(DEV), "e2m1")
    assert zeros is None and scales.shape == (2, 40, 12)
    c, b = R.quant_e2m1(w.double().numpy().reshape(80, 384))
    assert np.array_equal(scales.cpu().numpy().reshape(80, 12), b)
    assert np.array_equal(R.nibbles(codes.cpu().numpy()).reshape(80, 384), c)


@pytest.mark.parametrize("N,K,group", [(16, 128, 128), (33, 640, 32), (100, 1152, 64), (1, 512, 32), (48, 2048, 128)])
def test_preshuffle_int4(N, K, group):
    rng = np.random.default_rng(N)
    codes = rng.integers(0, 256, (N, K // 2), np.uint8)
    scales = bf16(rng, N, K // group)
    zeros = rng.integers(0, 16, (N, K // group), np.uint8)
    got = F.w4_preshuffle(dev(codes), scales.to(DEV), dev(zeros))
    ref = R.preshuffled(codes, scales.view(torch.int16).numpy(), zeros)
    assert np.array_equal(got[0].cpu().numpy(), ref[0])
    assert np.array_equal(got[1].cpu().view(torch.int16).numpy(), ref[1])
    assert np.array_equal(got[2].cpu().numpy(), ref[2])
    assert F.w4_preshuffle(dev(codes), scales.to(DEV))[2] is None


@pytest.mark.parametrize("N,K", [(16, 128), (33, 640), (256, 1024)])
def test_preshuffle_e2m1(N, K):
    rng = np.random.default_rng(N)
    codes = rng.integers(0, 256, (3, N, K // 2), np.uint8)
    scales = rng.integers(1, 255, (3, N, K // 32), np.uint8)
    got = F.w4_preshuffle(dev(codes), dev(scales))
    for e in range(3):
        ref = R.preshuffled(codes[e], scales[e])
        assert np.array_equal(got[0][e].cpu().numpy(), ref[0]) and np.array_equal(got[1][e].cpu().numpy(), ref[1])


# ---------------------------------------------------------------- products with 4-bit weights

FORMATS = [("e2m1", 32, False), ("int4", 32, False), ("int4", 32, True), ("int4", 64, False), ("int4", 64, True),
           ("int4", 128, False), ("int4", 128, True)]


def weights_of(rng, N, K, format, group, zero_points):
    """Row-order weights, their values and sum-bound values |16 + c| + |16 + z| (or the values), and the laid out form."""
    codes = rng.integers(0, 256, (N, K // 2), np.uint8)
    zeros = None
    if format == "e2m1":
        scales = rng.integers(117, 123, (N, K // 32), np.uint8)
        values = R.w4_values(codes, scales)
        size = np.abs(values)
        s = dev(scales)
    else:
        s = (bf16(rng, N, K // group).abs() + 0.01).to(DEV)
        zeros = rng.integers(0, 16, (N, K // group), np.uint8) if zero_points else None
        sv = R.bf16_values(s)
        values = R.w4_values(codes, sv, zeros)
        z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, 1)
        size = (32.0 + R.nibbles(codes) + z) * np.repeat(sv, group, 1)
    laid = F.w4_preshuffle(dev(codes), s, None if zeros is None else dev(zeros))
    return values, size, laid


def within(got, ref, bound):
    over = np.abs(got - ref) > bound
    assert not over.any(), "%d of %d values over the bound, the first at %s" % (over.sum(), over.size, np.argwhere(over)[0])


def check_gemv(x, values, size, out):
    ref = R.bf16_values(x) @ values.T
    K = values.shape[1]
    # a group's sum is at most 128 additions deep, the groups' K / 32, the wavefronts' 16; each is off by 2^-24 of what
    # was summed, twice that where the matrix instruction cuts off
    bound = 2 * (128 + K / 32 + 16) * R.F32_U * (np.abs(R.bf16_values(x)) @ size.T)
    bound += R.BF16_U * (np.abs(ref) + bound)
    got = R.bf16_values(out)
    assert got.shape == ref.shape and np.isfinite(got).all()
    within(got, ref, bound)
    if ref.size > 4000:
        assert np.linalg.norm(got - ref) <= 0.6 * R.BF16_U * np.linalg.norm(ref)  # in the mean well under the largest


@pytest.mark.parametrize("format,group,zero_points", FORMATS)
@pytest.mark.parametrize("T,N,K", [(1, 512, 512), (1, 17, 128), (2, 100, 1152), (5, 1031, 2048), (16, 64, 4096),
                                   (17, 48, 640), (33, 100, 1024), (48, 32, 384), (64, 300, 512), (65, 31, 256),
                                   (200, 16, 1152)])
def test_gemv(format, group, zero_points, T, N, K):
    rng = np.random.default_rng([T, N, K, group])
    values, size, laid = weights_of(rng, N, K, format, group, zero_points)
    x = bf16(rng, T, K)
    x[:, ::37] *= 50
    out = poisoned(T, N)
    got = F.w4_group_gemv_nt(x.to(DEV), laid[0], laid[1], N, zeros=laid[2], out=out)
    assert got is out
    check_gemv(x, values, size, got)


@pytest.mark.parametrize("format,group,zero_points", FORMATS)
@pytest.mark.parametrize("T,N,K", [(3, 4112, 512), (6, 4113, 1152), (2, 5136, 640), (7, 5137, 512), (8, 5121, 384), (16, 4200, 640), (20, 4099, 512), (40, 4128, 640),
                                   (64, 4111, 384), (4, 16400, 256), (5, 16384, 640), (16, 16401, 384), (17, 16384, 512),
                                   (33, 16500, 256), (64, 16385, 384), (70, 16384, 128), (5, 8208, 640),
                                   (16, 8500, 1152), (30, 10001, 256), (48, 8209, 384), (64, 16383, 128), (65, 9000, 1408)])
def test_gemv_of_many_rows(format, group, zero_points, T, N, K):
    """Two tiles a wavefront, and tokens shared through LDS."""
    test_gemv(format, group, zero_points, T, N, K)


@pytest.mark.parametrize("format,group,zero_points", FORMATS)
def test_gemv_integers(format, group, zero_points):
    """Sums that fp32 holds exactly: equal to the rounded sum bit for bit."""
    rng = np.random.default_rng(7)
    T, N, K = 19, 200, 1664
    codes = rng.integers(0, 256, (N, K // 2), np.uint8)
    zeros = rng.integers(0, 16, (N, K // group), np.uint8) if zero_points else None
    if format == "e2m1":
        scales = rng.integers(126, 130, (N, K // 32), np.uint8)
        s, sv = dev(scales), scales
    else:
        sv = np.exp2(rng.integers(-1, 3, (N, K // group))).astype(np.float64)
        s = R.round_bf16(sv).to(DEV)
    x = torch.from_numpy(rng.integers(-4, 5, (T, K)).astype(np.float32)).to(torch.bfloat16)
    laid = F.w4_preshuffle(dev(codes), s, None if zeros is None else dev(zeros))
    got = F.w4_group_gemv_nt(x.to(DEV), laid[0], laid[1], N, zeros=laid[2])
    ref = R.round_bf16(R.bf16_values(x) @ R.w4_values(codes, sv, zeros).T)
    assert torch.equal(got.cpu().view(torch.int16), ref.view(torch.int16))


def test_gemv_strided_and_views():
    rng = np.random.default_rng(3)
    T, N, K = 6, 70, 640
    values, size, laid = weights_of(rng, N, K, "int4", 64, True)
    wide = bf16(rng, T, K + 24)
    x = wide.to(DEV)[:, 8:8 + K]
    out = poisoned(T + 1, N + 11)
    F.w4_group_gemv_nt(x, laid[0], laid[1], N, zeros=laid[2], out=out[:T, 3:3 + N])
    check_gemv(wide[:, 8:8 + K], values, size, out[:T, 3:3 + N])
    assert out[T].isnan().all() and out[:, :3].isnan().all() and out[:, 3 + N:].isnan().all()


def test_gemv_empty():
    rng = np.random.default_rng(3)
    _, _, laid = weights_of(rng, 32, 256, "e2m1", 32, False)
    x = bf16(rng, 3, 256).to(DEV)
    assert F.w4_group_gemv_nt(x[:0], laid[0], laid[1], 32).shape == (0, 32)
    assert F.w4_group_gemv_nt(x, laid[0][:0], laid[1][:0], 0).shape == (3, 0)


def test_gemv_values_that_are_not_finite_stay_with_their_token():
    rng = np.random.default_rng(4)
    values, size, laid = weights_of(rng, 64, 512, "int4", 128, False)
    x = bf16(rng, 5, 512)
    clean = F.w4_group_gemv_nt(x.to(DEV), laid[0], laid[1], 64)
    x[2, 100] = float("nan")
    x[3, 7] = float("inf")
    got = F.w4_group_gemv_nt(x.to(DEV), laid[0], laid[1], 64)
    assert torch.equal(got[[0, 1, 4]], clean[[0, 1, 4]])
    assert got[2].isnan().all() and not got[3].isfinite().any()


# ---------------------------------------------------------------- mixture-of-experts layer

KINDS = ["plain", "preshuffled", "w4"]
CALL = {"plain": "moe_decode_layer", "preshuffled": "moe_decode_layer_preshuffled", "w4": "moe_decode_layer_w4"}


def e4m3(t):
    return t.view(torch.float8_e4m3fn).double().cpu().numpy()


class Layer:
    def __init__(self, rng, E, K, H, kind):
        self.kind, self.E, self.K, self.H = kind, E, K, H
        self.w = [self.product(rng, 2 * H, K), self.product(rng, K, H)]

    def product(self, rng, N, K):
        """(values [E, N, K], weights, scales) of one product, values about 1 / sqrt(K)."""
        E = self.E
        if self.kind == "w4":
            codes = rng.integers(0, 256, (E, N, K // 2), np.uint8)
            scales = rng.integers(-3, 1, (E, N, K // 32)) + 127 - int(np.log2(K) / 2)
            scales = scales.astype(np.uint8)
            c, s, _ = F.w4_preshuffle(dev(codes), dev(scales))
            return R.w4_values(codes, scales), c, s
        codes = torch.from_numpy(rng.standard_normal((E, N, K)).astype(np.float32) * 90).clamp(-448, 448).to(torch.float8_e4m3fn)
        scales = np.exp2(rng.integers(-8, -5, (E, N // 128, K // 128)) - int(np.log2(K) / 2)).astype(np.float32)
        values = codes.double().numpy() * np.repeat(np.repeat(scales.astype(np.float64), 128, 1), 128, 2)
        w = codes.view(torch.uint8).to(DEV)
        if self.kind == "preshuffled":
            w = torch.stack([F.fp8_weight_preshuffle(w[e]) for e in range(E)])
        return values, w, dev(scales)

    def __call__(self, q, sf, ids, weights, base=None, out=None, **kw):
        (_, w13, s13), (_, w2, s2) = self.w
        return getattr(F, CALL[self.kind])(q, sf, ids, weights, w13, s13, w2, s2, base=base, out=out, **kw)

    def reference(self, q, sf, ids, weights, base=None):
        T = q.shape[0]
        b = sf[:, :T].contiguous().cpu().numpy().view(np.uint8).reshape(-1, T, 4).transpose(1, 0, 2).reshape(T, -1)
        x = e4m3(q.contiguous()) * np.repeat(np.exp2(b[:, :self.K // 128].astype(np.float64) - 127), 128, 1)
        return R.moe_layer(x, ids.cpu().numpy(), weights.double().cpu().numpy(), self.w[0][0], self.w[1][0],
                           None if base is None else R.bf16_values(base))


def tokens(rng, T, K):
    return F.fp8_quant_group_pack(bf16(rng, T, K).to(DEV))


def check_layer(layer, got, args):
    ref, bound = layer.reference(*args)
    g = R.bf16_values(got)
    assert np.isfinite(g).all()
    within(g, ref, bound)
    if ref.size > 2000 and np.abs(ref).max() > 0:
        # a bf16 rounding is off by 2^-8 at most and, spread over a step of between 2^-8 and 2^-7 of the value, by 2^-9 in
        # the mean square; an activation that goes to the other code adds at most 2^-4 of itself, in one of 10^4 places
        assert np.linalg.norm(g - ref) <= (0.5 * R.BF16_U + 2.0 ** -4 * 0.02) * np.linalg.norm(ref)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,topk,K,H,base", [
    (1, 8, 2, 512, 256, True), (1, 4, 1, 128, 128, False), (2, 40, 8, 640, 384, True), (7, 3, 3, 1152, 128, False),
    (16, 16, 4, 512, 640, True), (17, 5, 2, 256, 1024, True), (33, 8, 2, 384, 256, False), (48, 2, 2, 256, 128, True),
    (64, 8, 5, 512, 384, True), (64, 1, 1, 128, 256, False), (1, 64, 64, 256, 256, False), (3, 1000, 20, 128, 128, True),
    (20, 5, 2, 640, 640, True), (30, 200, 4, 128, 256, False), (64, 4, 1, 256, 1152, True), (16, 16, 4, 2048, 2048, False),
    (9, 8, 7, 1152, 640, True), (1, 4, 2, 4224, 1152, True), (2, 8, 8, 4224, 256, False), (12, 12, 5, 4352, 128, True),
    (24, 4, 2, 4224, 128, False), (40, 6, 3, 4352, 256, True), (64, 2, 1, 4224, 128, False), (1, 16, 12, 640, 2048, True)])
def test_layer(kind, T, E, topk, K, H, base):
    rng = np.random.default_rng([T, E, topk, K, H])
    layer = Layer(rng, E, K, H, kind)
    q, sf = tokens(rng, T, K)
    ids = dev(np.stack([rng.permutation(E)[:topk] for _ in range(T)]).astype(np.int32))
    weights = dev(rng.random((T, topk)).astype(np.float32) - 0.2)
    args = (q, sf, ids, weights, bf16(rng, T, K).to(DEV) if base else None)
    out = poisoned(T, K)
    assert layer(*args, out=out) is out
    check_layer(layer, out, args)


@pytest.mark.parametrize("kind", KINDS)
def test_layer_pairs_that_are_left_out(kind):
    """Ids outside the experts, tokens without any, an expert named twice, and experts nobody names."""
    rng = np.random.default_rng(5)
    T, E, topk, K, H = 20, 12, 3, 512, 256
    layer = Layer(rng, E, K, H, kind)
    q, sf = tokens(rng, T, K)
    ids = rng.integers(0, 5, (T, topk)).astype(np.int32)
    ids[3] = -1
    ids[4] = [E, 1 << 30, -(1 << 31)]
    ids[5] = 2
    ids[6] = [7, -1, 7]
    ids[7] = [-1, 0, E + 3]
    weights = dev(rng.random((T, topk)).astype(np.float32))
    base = bf16(rng, T, K).to(DEV)
    for b in (base, None):
        args = (q, sf, dev(ids), weights, b)
        got = layer(*args)
        check_layer(layer, got, args)
        for t in (3, 4):
            assert torch.equal(got[t], torch.zeros_like(got[t]) if b is None else b[t])


@pytest.mark.parametrize("kind", KINDS)
def test_layer_of_nothing(kind):
    rng = np.random.default_rng(6)
    layer = Layer(rng, 4, 256, 128, kind)
    q, sf = tokens(rng, 3, 256)
    ids, weights = torch.full((3, 2), -1, dtype=torch.int32, device=DEV), torch.ones(3, 2, device=DEV)
    assert not layer(q, sf, ids, weights).any()
    assert layer(q[:0], sf, ids[:0], weights[:0]).shape == (0, 256)


def test_layer_integers():
    """gate = 32 (its silu in fp32 is 32), up and down small integers: equal to the rounded sum bit for bit."""
    rng = np.random.default_rng(8)
    T, E, topk, K, H = 21, 6, 3, 384, 256
    x = rng.integers(-1, 2, (T, K)).astype(np.float32)
    x[:, 0] = 4
    q = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    sf = torch.full((1, T + 3), 0x7F7F7F7F, dtype=torch.int32, device=DEV)
    up = np.zeros((E, H, K), np.float32)
    for e in range(E):
        for h in range(H):
            up[e, h, rng.choice(np.arange(1, K), 6, replace=False)] = rng.choice([-1, 1], 6)
    gate = np.zeros((E, H, K), np.float32)
    gate[:, :, 0] = 8
    w2 = rng.integers(-2, 3, (E, K, H)).astype(np.float32)
    w13 = np.concatenate([gate, up], 1)

    def codes(w):
        return torch.from_numpy(w).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    ids = dev(np.stack([rng.permutation(E)[:topk] for _ in range(T)]).astype(np.int32))
    weights = dev(np.exp2(rng.integers(-2, 2, (T, topk))).astype(np.float32))
    base = torch.from_numpy(rng.integers(-50, 50, (T, K)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    ones = [torch.ones(E, 2 * H // 128, K // 128, device=DEV), torch.ones(E, K // 128, H // 128, device=DEV)]
    out = base.double().cpu().numpy()
    for t in range(T):
        for j in range(topk):
            e = int(ids[t, j])
            y = 32.0 * (up[e].astype(np.float64) @ x[t])
            assert np.abs(y).max() <= 448
            out[t] += float(weights[t, j]) * (w2[e].astype(np.float64) @ y)
    ref = R.round_bf16(out)
    for name in ("moe_decode_layer", "moe_decode_layer_preshuffled"):
        a, b = codes(w13), codes(w2)
        if name.endswith("preshuffled"):
            a, b = (torch.stack([F.fp8_weight_preshuffle(w[e]) for e in range(E)]) for w in (a, b))
        got = getattr(F, name)(q, sf, ids, weights, a, ones[0], b, ones[1], base=base)
        assert torch.equal(got.cpu().view(torch.int16), ref.view(torch.int16)), name
    # the same weights are values of e2m1 too (8 is not: 4 under a scale of 2)
    def four(w, byte):
        n = np.zeros(w.shape, np.int64)
        for v, c in ((0, 0), (1, 2), (2, 4), (4, 6)):
            n[np.abs(w) == v] = c
        n += 8 * (w < 0)
        return F.w4_preshuffle(dev(R.packed(n)), dev(np.full((*w.shape[:-1], w.shape[-1] // 32), byte, np.uint8)))
    g = np.concatenate([gate / 2, up], 1)
    c13, s13, _ = four(g, 127)
    s13 = s13.clone()
    s13[:, :H // 16] += 1
    c2, s2, _ = four(w2, 127)
    got = F.moe_decode_layer_w4(q, sf, ids, weights, c13, s13, c2, s2, base=base)
    assert torch.equal(got.cpu().view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("kind", KINDS)
def test_layer_strided(kind):
    rng = np.random.default_rng(9)
    T, E, topk, K, H = 5, 4, 2, 640, 256
    layer = Layer(rng, E, K, H, kind)
    q, sf = tokens(rng, T, K)
    wide = torch.zeros(T, K + 48, dtype=torch.uint8, device=DEV)
    wide[:, 16:16 + K] = q
    sfw = torch.full((sf.shape[0], T + 9), 0x55555555, dtype=torch.int32, device=DEV)
    sfw[:, :T] = sf[:, :T]
    ids = dev(np.stack([rng.permutation(E)[:topk] for _ in range(T)]).astype(np.int32))
    weights = dev(rng.random((T, topk)).astype(np.float32))
    base = bf16(rng, T, K + 16).to(DEV)
    out = poisoned(T + 1, K + 8)
    layer(wide[:, 16:16 + K], sfw, ids, weights, base=base[:, 8:8 + K], out=out[:T, :K])
    check_layer(layer, out[:T, :K], (q, sf, ids, weights, base[:, 8:8 + K]))
    assert out[T].isnan().all() and out[:, K:].isnan().all()


@pytest.mark.parametrize("kind", KINDS)
def test_layer_values_that_are_not_finite(kind):
    """NaN and infinity in one token, in an expert's weights and in a routing weight stay where the formula has them."""
    rng = np.random.default_rng(10)
    T, E, topk, K, H = 18, 4, 2, 256, 128
    layer = Layer(rng, E, K, H, kind)
    q, sf = tokens(rng, T, K)
    ids = np.stack([rng.permutation(3)[:topk] for _ in range(T)]).astype(np.int32)
    ids[11] = [0, 3]
    ids[12] = [3, -1]
    weights = rng.random((T, topk)).astype(np.float32)
    clean = layer(q, sf, dev(ids), dev(weights))
    q = q.clone()
    q[2, 5] = 0x7F  # the NaN code
    weights[3, 1] = np.inf
    got = layer(q, sf, dev(ids), dev(weights))
    same = [t for t in range(T) if t not in (2, 3)]
    assert torch.equal(got[same], clean[same])
    assert got[2].isnan().all() and not got[3].isfinite().any()
    if kind != "w4":  # e2m1 has no such code
        w2 = layer.w[1][1]
        kept = w2[3].clone()
        w2[3] = 0x7F
        got = layer(q, sf, dev(ids), dev(weights))
        same = [t for t in same if t not in (11, 12)]
        assert torch.equal(got[same], clean[same]) and got[[11, 12]].isnan().all()
        w2[3] = kept


@pytest.mark.parametrize("T,topk", [(2, 3), (30, 4)])
def test_layer_weights_of_pairs_left_out_do_not_matter(T, topk):
    rng = np.random.default_rng(12)
    layer = Layer(rng, 5, 256, 128, "preshuffled")
    q, sf = tokens(rng, T, 256)
    ids = rng.integers(-2, 7, (T, topk)).astype(np.int32)
    weights = rng.random((T, topk)).astype(np.float32)
    clean = layer(q, sf, dev(ids), dev(weights))
    weights[(ids < 0) | (ids >= 5)] = np.nan
    assert torch.equal(layer(q, sf, dev(ids), dev(weights)), clean) and clean.isfinite().all()


@pytest.mark.parametrize("kind", ["plain", "preshuffled"])
def test_layer_reads_the_exponent_of_block_scales(kind):
    """As every product of UE8M0 scales: 2^floor(log2 |s|)."""
    rng = np.random.default_rng(13)
    layer = Layer(rng, 4, 384, 256, kind)
    q, sf = tokens(rng, 6, 384)
    ids, weights = dev(rng.integers(0, 4, (6, 2)).astype(np.int32)), dev(rng.random((6, 2)).astype(np.float32))
    clean = layer(q, sf, ids, weights)
    for _, _, s in layer.w:
        s.mul_(-1.75)
    assert torch.equal(layer(q, sf, ids, weights), clean)


def test_scale_words_past_the_columns_do_not_matter():
    """Bytes of groups past K, and scale words of another token, may hold anything."""
    rng = np.random.default_rng(11)
    layer = Layer(rng, 3, 640, 128, "plain")
    q, sf = tokens(rng, 4, 640)
    ids, weights = dev(rng.integers(0, 3, (4, 1)).astype(np.int32)), torch.ones(4, 1, device=DEV)
    clean = layer(q, sf, ids, weights)
    sf = sf.clone()
    sf[1] |= torch.tensor(-256, dtype=torch.int32, device=DEV)  # 0xFFFFFF00: the bytes of groups 5..7
    assert torch.equal(layer(q, sf, ids, weights), clean)
