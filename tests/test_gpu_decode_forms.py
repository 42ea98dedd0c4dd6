"""The operators of a decode step in every form that their sizes choose: values against references in 64 bits, values that
are not finite, and the ways of calling them (tests/test_decode_forms.py checks that no kernel is left out)."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_token_amd as F
import decode_reference as R
import test_gpu_decode_calls as calls
import test_gpu_decode_ops as ops
from test_gpu_decode_ops import DEV, FORMATS, KINDS, Layer, bf16, dev, tokens, weights_of

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


@pytest.mark.parametrize("T,N", [(1, 16), (6, 5152), (20, 32), (20, 8224), (6, 16400)])
@pytest.mark.parametrize("byte,most", [(1, 7), (2, 7), (251, 7), (252, 7), (253, 5), (254, 3)])
def test_gemv_e2m1_scales_at_their_ends(byte, most, T, N):
    """Every code whose value is under 2^128, a code a row: sums of one power of two are exact."""
    K = 128
    codes = np.resize(np.concatenate([np.arange(most + 1), 8 + np.arange(most + 1)]), N).astype(np.uint8)
    laid = F.w4_preshuffle(dev(np.repeat(17 * codes[:, None], K // 2, 1)), dev(np.full((N, K // 32), byte, np.uint8)))
    e = max(-120, min(120, 127 - byte))
    got = F.w4_group_gemv_nt(torch.full((T, K), 2.0 ** e, dtype=torch.bfloat16, device=DEV), laid[0], laid[1], N)
    want = K * R.E2M1[codes] * 2.0 ** (e + byte - 127)
    assert (got.double().cpu().numpy() == want).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,N", [(1, 64), (7, 5137), (20, 48), (40, 4128), (20, 8208)])
def test_gemv_zero_points_of_a_byte(group, T, N):
    """Zero points up to 255, in sums that fp32 holds exactly: 640 * 4 * 255 of tokens up to 4, under scales of 1/2 to 4."""
    rng = np.random.default_rng([T, N, group])
    K = 640
    codes, zeros = rng.integers(0, 256, (N, K // 2), np.uint8), rng.integers(0, 256, (N, K // group)).astype(np.uint8)
    sv = np.exp2(rng.integers(-1, 3, (N, K // group))).astype(np.float64)
    laid = F.w4_preshuffle(dev(codes), R.round_bf16(sv).to(DEV), dev(zeros))
    x = torch.from_numpy(rng.integers(-4, 5, (T, K)).astype(np.float32)).to(torch.bfloat16)
    got = F.w4_group_gemv_nt(x.to(DEV), laid[0], laid[1], N, zeros=laid[2])
    want = R.round_bf16(R.bf16_values(x) @ R.w4_values(codes, sv, zeros).T)
    assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))


def e4m3_code(value):
    return torch.tensor(value).to(torch.float8_e4m3fn).view(torch.uint8).item()


@pytest.mark.parametrize("T", [1, 20, 40])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("where", ["up", "down", "tokens"])
@pytest.mark.parametrize("end", ["low", "high"])
def test_layer_scales_at_their_ends(where, end, kind, T):
    """One product of powers of two a column, so that the layer's output is exact: gate 32 (its silu in fp32 is 32), up and
    down one weight each, under the smallest and largest scales that bf16 holds every code of."""
    K = H = 128
    w4 = kind == "w4"
    lo, hi = (-126, 125) if w4 and where != "tokens" else (-124, 119)
    codes = [0.5, 1.0, 6.0] if w4 and where != "tokens" else [2.0 ** -9, 1.0, 448.0]
    s = lo if end == "low" else hi
    # exponents of the scales of the tokens, the gate's weights (their code is 1), the up product's and the down product's
    t = {"up": max(-100, min(100, -s)), "down": 0, "tokens": s}[where]
    gate = 5 - 8 - t  # the tokens' code for the gate is 256
    up = {"up": s, "down": -30 if s > 0 else 0, "tokens": max(-100, min(100, -s))}[where]
    down = s if where == "down" else 0
    for code in codes:
        u, d, x = (code if where == n else 1.0 for n in ("up", "down", "tokens"))
        q = torch.zeros(T, K, dtype=torch.uint8, device=DEV)
        q[:, 0], q[:, 1] = e4m3_code(256.0), e4m3_code(x)
        sf = torch.full((1, T), 127 + t, dtype=torch.int32, device=DEV)
        w13, w2 = np.zeros((1, 2 * H, K)), np.zeros((1, K, H))
        w13[:, :H, 0], w13[:, H:, 1], w2[:, :, 0] = 1.0, u, d
        e13 = np.repeat(np.array([gate, up]), H)
        if w4:
            def four(w, e):
                n = np.abs(w[..., None] - R.E2M1[:8]).argmin(-1)
                b = np.repeat((127 + e).astype(np.uint8)[None, :, None], w.shape[2] // 32, 2)
                return F.w4_preshuffle(dev(R.packed(n)), dev(b))[:2]
            args = *four(w13, e13), *four(w2, np.full(K, down))
        else:
            def eight(w):
                c = torch.from_numpy(w).float().to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
                return c if kind == "plain" else torch.stack([F.fp8_weight_preshuffle(c[0])])
            args = (eight(w13), torch.tensor([[[2.0 ** gate], [2.0 ** up]]], device=DEV), eight(w2),
                    torch.full((1, 1, 1), 2.0 ** down, device=DEV))
        got = getattr(F, ops.CALL[kind])(q, sf, torch.zeros(T, 1, dtype=torch.int32, device=DEV),
                                         torch.ones(T, 1, device=DEV), *args)
        want = 32.0 * u * x * 2.0 ** (t + up) * d * 2.0 ** down
        assert (got.double() == want).all(), (code, want, got[0, :2])


#: tokens, choices, experts, hidden and half size of a layer in each form: K in four parts and in two; then up to 64 pairs
#: and more, by 16, 32 and 64 tokens, with 16 and with 32 output columns a workgroup
LAYER_FORMS = [(1, 2, 6, 512, 256), (1, 48, 48, 256, 256)] + [
    (T, topk, 4, K, H) for K in (512, 4224) for T, topk, H in (
        (16, 4, 640), (20, 3, 128), (40, 1, 128), (16, 5, 128), (24, 4, 128), (40, 3, 128))]
#: a product in each form of tiles and tokens
GEMV_FORMS = [(1, 100), (7, 300), (14, 100), (20, 100), (40, 100), (64, 100), (3, 5200), (6, 5200), (14, 4200), (20, 4200),
              (40, 4200), (64, 4200), (6, 9000), (20, 9000), (40, 9000), (64, 9000), (6, 16400), (20, 16400), (40, 16400),
              (64, 16400)]


def layers(rng, kind):
    out = []
    for T, topk, E, K, H in LAYER_FORMS:
        layer = Layer(rng, E, K, H, kind)
        q, sf = tokens(rng, T, K)
        ids, w = dev(rng.integers(0, E, (T, topk)).astype(np.int32)), dev(rng.random((T, topk)).astype(np.float32))
        base = bf16(rng, T, K).to(DEV)
        out.append((lambda o, a=(layer, q, sf, ids, w, base), **kw: a[0](*a[1:], out=o, **kw), (T, K)))
    return out


def products(rng, kind):
    out = []
    for i, (T, N) in enumerate(GEMV_FORMS):
        _, _, laid = weights_of(rng, N, 640, *FORMATS[i % len(FORMATS)])
        x = bf16(rng, T, 640).to(DEV)
        out.append((lambda o, a=(x, laid, N), **kw: F.w4_group_gemv_nt(a[0], a[1][0], a[1][1], a[2], zeros=a[1][2], out=o, **kw),
                    (T, N)))
    return out


@pytest.mark.parametrize("way", ["test_named_streams", "test_calls_beside_each_other", "test_captured_and_replayed"])
@pytest.mark.parametrize("kind", KINDS + ["products"])
def test_ways_of_calling(monkeypatch, kind, way):
    monkeypatch.setattr(calls, "works", lambda rng: (products if kind == "products" else layers)(rng, kind))
    getattr(calls, way)()


@pytest.mark.parametrize("kind", KINDS)
def test_experts_past_32_bits(kind):
    """The last experts of weights past 2^31 bytes, against a copy of them that has as many experts as the call has pairs: the
    same kernels with the same order of sums, so equal bits."""
    T, topk, K, H = 3, 2, 7168, 2048
    pairs = T * topk
    E = 220 if kind == "w4" else 120
    rng = np.random.default_rng(15)
    q, sf = tokens(rng, T, K)
    g = torch.Generator(device=DEV).manual_seed(3)

    def codes(*shape):  # finite e4m3, or any e2m1
        c = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
        return c if kind == "w4" else c & 0xF7
    if kind == "w4":
        w13, w2 = codes(E, 2 * H // 16, K // 128, 1024), codes(E, K // 16, H // 128, 1024)
        s13, s2 = (torch.full(s, 117, dtype=torch.uint8, device=DEV) for s in ((E, 2 * H // 16, 14, 64, 4), (E, K // 16, 4, 64, 4)))
    else:
        w13, w2 = codes(E, 2 * H, K), codes(E, K, H)
        s13, s2 = (torch.full(s, 2.0 ** -13, device=DEV) for s in ((E, 2 * H // 128, K // 128), (E, K // 128, H // 128)))
    assert w13.numel() > 1 << 31
    ids = dev(np.stack([E - pairs + rng.permutation(pairs)[:topk] for _ in range(T)]).astype(np.int32))
    ids[0, 0] = E - 1
    w = torch.rand(T, topk, generator=g, device=DEV)
    call = getattr(F, ops.CALL[kind])
    got = call(q, sf, ids, w, w13, s13, w2, s2)
    want = call(q, sf, ids - (E - pairs), w, *(t[-pairs:].contiguous() for t in (w13, s13, w2, s2)))
    assert got.isfinite().all() and got.abs().max() > 0 and torch.equal(got, want)
    del w13, w2
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,topk,K,H,base", [(1, 1, 1, 65536, 128, True), (20, 1, 1, 65536, 128, False),
                                               (3, 1, 1, 128, 65536, False), (33, 1, 2, 128, 65536, True)])
def test_layer_of_the_largest_sizes(kind, T, E, topk, K, H, base):
    rng = np.random.default_rng([T, K])
    layer = Layer(rng, E, K, H, kind)
    q, sf = tokens(rng, T, K)
    ids, weights = np.zeros((T, topk), np.int32), dev(rng.random((T, topk)).astype(np.float32))
    ids[:, 1:] = -1
    args = (q, sf, dev(ids), weights, bf16(rng, T, K).to(DEV) if base else None)
    ops.check_layer(layer, layer(*args), args)


@pytest.mark.parametrize("format,group,zero_points", FORMATS)
@pytest.mark.parametrize("T,N,K", [(2, 20, 65536), (20, 16, 65536), (64, 16, 65536)])
def test_gemv_of_the_largest_k(format, group, zero_points, T, N, K):
    ops.test_gemv(format, group, zero_points, T, N, K)


@pytest.mark.parametrize("T,N", [(6, 8208), (40, 16400)])
def test_gemv_through_lds_of_the_largest_k(T, N):
    """Against the same rows of weights in a product of few, in sums that are exact: under 2 * 32 * 65536 = 2^22."""
    K = 65536
    g = torch.Generator(device=DEV).manual_seed(4)
    codes = torch.randint(0, 256, (-(-N // 16), K // 128, 1024), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.ones(-(-N // 16), K // 512, 16, 4, dtype=torch.bfloat16, device=DEV)
    x = torch.randint(-2, 3, (T, K), generator=g, device=DEV).to(torch.bfloat16)
    got = F.w4_group_gemv_nt(x, codes, scales, N)
    for at in (0, 200, N // 16 - 4):
        want = F.w4_group_gemv_nt(x, codes[at:at + 4].contiguous(), scales[at:at + 4].contiguous(), 64)
        assert torch.equal(got[:, 16 * at:16 * at + 64], want)
    del codes
    torch.cuda.empty_cache()


def far_apart(t, ld):
    """t's rows, ld elements from one to the next."""
    wide = torch.empty(t.shape[0] * ld, dtype=t.dtype, device=DEV).view(t.shape[0], ld)[:, :t.shape[1]]
    wide.copy_(t)
    return wide


@pytest.mark.parametrize("T,topk", [(64, 2), (33, 1), (3, 2)])
def test_layer_of_rows_far_apart(T, topk):
    """Rows of q and of the scale words that span nearly 2 GiB, as far as the layer takes them, and rows of base and out past
    2^32 elements."""
    rng = np.random.default_rng(T)
    K = 640
    layer = Layer(rng, 4, K, 256, "plain")
    q, sf = tokens(rng, T, K)
    ids, w = dev(rng.integers(0, 4, (T, topk)).astype(np.int32)), dev(rng.random((T, topk)).astype(np.float32))
    base = bf16(rng, T, K).to(DEV)
    want = layer(q, sf, ids, w, base=base)
    ldq = ((1 << 31) // T - K) // 16 * 16
    ld = ((1 << 32) // (T - 1) // 8 + 1) * 8
    out = far_apart(torch.zeros(T, K, dtype=torch.bfloat16, device=DEV), ld)
    got = layer(far_apart(q, ldq), far_apart(sf[:, :T], (1 << 29) - 128), ids, w, base=far_apart(base, ld), out=out)
    assert got is out and torch.equal(got, want)
    del got, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,N", [(3, 100), (64, 100), (40, 8208), (130, 100)])
def test_gemv_of_rows_far_apart(T, N):
    """64 rows of x that span nearly 2 GiB, and rows of out past 2^32 elements."""
    rng = np.random.default_rng(T)
    K = 640
    _, _, laid = weights_of(rng, N, K, "int4", 64, True)
    x = bf16(rng, T, K).to(DEV)
    want = F.w4_group_gemv_nt(x, laid[0], laid[1], N, zeros=laid[2])
    ldx = ((1 << 30) // min(T, 64) - K) // 8 * 8
    out = far_apart(torch.zeros(T, N, dtype=torch.bfloat16, device=DEV), (1 << 32) // (T - 1) + N)
    got = F.w4_group_gemv_nt(far_apart(x, ldx), laid[0], laid[1], N, zeros=laid[2], out=out)
    assert got is out and torch.equal(got, want)
    del got, out
    torch.cuda.empty_cache()


def made(w, format, group, zero_points, **kw):
    """w in 4 bits, in row order and laid out."""
    rows = F.w4_group_quant(w, format, group, zero_points, **kw)
    return [t for t in (*rows, *F.w4_preshuffle(*rows, **kw)) if t is not None]


@pytest.mark.parametrize("format,group,zero_points", [("e2m1", 32, False), ("int4", 64, True)])
def test_weights_past_32_bits(format, group, zero_points):
    """Past 2^32 values: the first and the last matrix against the same alone."""
    E, N, K = 520, 4096, 2048
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(6)
    some = torch.randn(4, N, K, generator=g, device=DEV).to(torch.bfloat16)
    for e in range(E):
        w[e] = some[e % 4]
    assert w.numel() > 1 << 32
    got = made(w, format, group, zero_points)
    for e in (0, E // 2, E - 1):
        for a, b in zip(got, made(w[e:e + 1], format, group, zero_points)):
            assert torch.equal(a[e], b[0])
    del w, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("format,group,zero_points", [("e2m1", 32, False), ("int4", 128, False), ("int4", 32, True)])
def test_weights_on_streams_and_in_graphs(format, group, zero_points):
    rng = np.random.default_rng(16)
    ws = [bf16(rng, 3, 50, 1152, std=0.05).to(DEV) for _ in range(2)]
    wants = [made(w, format, group, zero_points) for w in ws]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ws]
    for _ in range(4):
        got = []
        for w, s in zip(ws, streams):
            got.append(made(w, format, group, zero_points, stream=s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, wants) for a, b in zip(g, w))
    w = ws[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = made(w, format, group, zero_points)
    for turn in range(4):
        w.copy_(ws[turn % 2])
        for o in outs:
            o.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = made(ws[(turn + 1) % 2], format, group, zero_points)
        assert all(torch.equal(a, b) for a, b in zip(outs, wants[turn % 2])), turn
        assert all(torch.equal(a, b) for a, b in zip(eager, wants[(turn + 1) % 2]))
