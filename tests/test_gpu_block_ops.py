"""Routing, combine, residual norms and the 8-bit activation checkpoint on the GPU against
references in 64 bits (tests/block_reference.py), forward and backward.

Tolerances follow from the arithmetic: an output rounded once to bf16 is within 2^-8 of its
value, and an fp32 sum of n terms is within n * 2^-24 of the sum of their magnitudes; where a
bound below has a factor, its comment counts the roundings."""
import math

import numpy as np
import pytest
import torch

import block_reference as R
import block_scaled_fp8_token_amd as F
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rng(*seed):
    return np.random.default_rng([20, *seed])


def bf(a):
    """float64 array -> (bf16 device tensor, its values in 64 bits)."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(BF)
    return t.to(DEV), t.double().numpy()


def f32(a):
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32))
    return t.to(DEV), t.double().numpy()


def host(t):
    return t.detach().double().cpu().numpy()


def nans(*shape, dtype=BF):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def close(got, ref, bound, what=""):
    got = host(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), "%s: %d of %d off, first %s: %s for %s" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0].tolist(), got[bad][0], ref[bad][0])


def strided(t, extra):
    """The same values as rows of a wider tensor whose other columns are NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


# ------------------------------------------------------------------ routing

ROUTES = [  # T, E, topk, groups, topk_groups, group_top, scoring, bias, dtype
    (1, 1, 1, 1, 1, 1, "softmax", False, BF),
    (3, 5, 5, 1, 1, 1, "sigmoid", True, torch.float32),
    (9, 60, 6, 1, 1, 1, "softmax", False, BF),
    (64, 64, 8, 8, 3, 1, "softmax", False, torch.float32),
    (5, 72, 7, 9, 4, 2, "sigmoid", True, BF),
    (33, 160, 6, 8, 3, 1, "softmax", False, torch.float32),
    (40, 256, 8, 8, 4, 2, "sigmoid", True, torch.float32),
    (17, 256, 8, 8, 4, 2, "sigmoid", False, torch.float32),
    (13, 256, 8, 4, 2, 2, "softmax", False, torch.float32),
    (12, 96, 4, 1, 1, 1, "softmax", True, torch.float32),
    (6, 513, 3, 1, 1, 1, "sigmoid", True, torch.float32),
    (4, 1024, 64, 64, 8, 2, "sigmoid", True, torch.float32),
    (7, 384, 8, 1, 1, 1, "sigmoid", True, torch.float32),
    (5, 448, 7, 16, 5, 2, "sigmoid", True, torch.float32),
    (6, 512, 8, 1, 1, 1, "softmax", False, BF),
    (9, 40, 9, 1, 1, 1, "softmax", False, torch.float32),
]


def route_inputs(i, T, E, bias, dtype, masked=False):
    """Logits on a grid of 1/16 (exact in bf16, with ties), the bias in steps of 1/8."""
    g = rng(1, i, int(masked))
    l = np.clip(np.round(g.normal(size=(T, E)) * 24) / 16, -7, 7)
    if masked:
        l[g.random((T, E)) < 0.3] = -np.inf
        l[g.random((T, E)) < 0.05] = np.nan
        l[0] = -np.inf
        if T > 1:
            l[1, 1:] = np.nan
            l[1, 0] = 0.5
        if T > 2:
            l[2, E // 2] = np.inf
    b = g.integers(-4, 5, E) / 8.0 if bias else None
    return l, b


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("i", range(len(ROUTES)))
@pytest.mark.parametrize("renormalize", [True, False])
def test_route(i, renormalize, masked):
    T, E, k, G, kg, top, scoring, bias, dtype = ROUTES[i]
    l, b = route_inputs(i, T, E, bias, dtype, masked)
    opts = dict(groups=G, topk_groups=kg, group_top=top, scoring=scoring, renormalize=renormalize, scale=2.5)
    ids, w, gap = R.route(l, k, bias=b, **opts)
    assert gap > 1e-6  # so that fp32 (scores within 4 * 2^-24 of theirs) orders the ranks alike
    lt = torch.from_numpy(l).to(dtype).to(DEV)
    got_ids, got_w = F.moe_route_topk(strided(lt, 3), k, bias=None if b is None else f32(b)[0], **opts)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    # exp, sum of E, division, sum of k, division, scale: E + k + 16 roundings at the most
    close(got_w, w, (E + k + 16) * R.F32_U * np.abs(w) + 1e-37)


def test_route_ties_go_to_the_lowest():
    l = torch.zeros(2, 200, device=DEV)
    l[1, 150:] = 1.0
    ids, w = F.moe_route_topk(l, 8, scoring="sigmoid")
    assert ids.tolist() == [list(range(8)), list(range(150, 158))]
    assert torch.equal(w, torch.full_like(w, 0.125))
    ids, _ = F.moe_route_topk(l, 8, groups=8, topk_groups=2, group_top=2, scoring="sigmoid")  # tied groups: the lowest
    assert ids.tolist() == [list(range(8)), list(range(150, 158))]
    # saturated sigmoids tie as scores; without a bias the logits still rank
    l = torch.tensor([[30.0, 40.0, 35.0, 50.0]], device=DEV)
    assert F.moe_route_topk(l, 2, scoring="sigmoid")[0].tolist() == [[3, 1]]
    assert F.moe_route_topk(l, 2, bias=torch.zeros(4, device=DEV), scoring="sigmoid")[0].tolist() == [[0, 1]]


def test_route_extreme_logits():
    # chosen logits far under the largest (their group lost), and sums that underflow
    l = torch.full((1, 8), -200.0, device=DEV)
    l[0, 0] = 100.0
    b = torch.zeros(8, device=DEV)
    b[0] = -1e30
    ids, w = F.moe_route_topk(l, 2, bias=b, scoring="softmax")
    assert ids.tolist() == [[1, 2]] and torch.equal(w, torch.full_like(w, 0.5))
    ids, w = F.moe_route_topk(l - 100, 2, bias=b, scoring="sigmoid")  # both scores are 0: no weight, no NaN
    assert torch.equal(w, torch.zeros_like(w))
    l = torch.tensor([[3e38, 3.4e38, float("inf"), -3e38]], device=DEV)
    ids, w = F.moe_route_topk(l, 2, scoring="softmax")
    assert ids.tolist() == [[2, 1]] and w.isfinite().all()
    b = torch.tensor([0.0, float("nan"), float("-inf"), 0.0], device=DEV)
    assert F.moe_route_topk(l, 3, bias=b, scoring="sigmoid")[0].tolist() == [[0, 3, -1]]


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("k", [2, 9])  # either kernel
def test_route_masks_of_the_lowest_value(scoring, dtype, k):
    low = torch.finfo(dtype).min
    l = torch.full((3, 32), low, dtype=dtype, device=DEV)  # finite: every expert is available
    l[1, 7] = 1.0
    l[2, 4], l[2, 9] = torch.finfo(dtype).max, 0.0
    for renormalize in (True, False):
        ids, w = F.moe_route_topk(l, k, scoring=scoring, renormalize=renormalize)
        want = [top + [e for e in range(32) if e not in top] for top in ([], [7], [4, 9])]
        assert ids.tolist() == [row[:k] for row in want]
        assert w.isfinite().all()
        assert float(w[1, 0]) == pytest.approx(1.0 if renormalize or scoring == "softmax" else 1 / (1 + math.exp(-1)))
        assert not w[1, 1:].any()  # what a mask of the lowest value leaves has no weight


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, torch.float32), (5, 60, 6, BF), (9, 160, 2, torch.float32),
                                         (3, 256, 8, torch.float32), (2, 700, 64, torch.float32)])
def test_route_backward(T, E, k, dtype, scoring, renormalize):
    g = rng(2, E)
    l = torch.from_numpy(np.clip(g.normal(size=(T, E)) * 1.5, -6, 6)).to(dtype)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    dw = torch.from_numpy(g.normal(size=(T, k)).astype(np.float32))
    got = F.moe_route_topk_backward(strided(l.to(DEV), 5), torch.from_numpy(ids).int().to(DEV), dw.to(DEV),
                                    scoring=scoring, renormalize=renormalize, scale=1.75, d_logits=nans(T, E, dtype=dtype))
    # the formula, by automatic differentiation in 64 bits
    ld = l.double().requires_grad_(True)
    s = torch.sigmoid(ld) if scoring == "sigmoid" else torch.softmax(ld, 1)
    w = s.gather(1, torch.from_numpy(ids))
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    ref = torch.autograd.grad((w * dw.double()).sum() * 1.75, ld)[0].numpy()
    # each gradient is a product with a difference of dw and a mean of dw: magnitude 2 c max|dw| max(w)
    scale = 2 * 1.75 * float(dw.abs().max()) * w.detach().numpy().max(1, keepdims=True)
    bound = (E + 2 * k + 24) * R.F32_U * scale + (R.BF16_U * np.abs(ref) if dtype == BF else 0)
    close(got, ref, bound)
    # and differences of the forward formula
    eps, l64, d64 = 1e-5, l.double().numpy(), dw.double().numpy()
    for t, e in [(0, 0), (T - 1, E - 1), (T // 2, int(ids[T // 2, 0]))]:
        lp, lm = l64.copy(), l64.copy()
        lp[t, e] += eps
        lm[t, e] -= eps
        diff = ((R.route_weights(lp, ids, scoring, renormalize, 1.75) -
                 R.route_weights(lm, ids, scoring, renormalize, 1.75)) * d64).sum() / (2 * eps)
        assert abs(float(got[t, e]) - diff) <= float(bound[t, 0] if bound.shape[1] == 1 else bound[t, e]) + 1e-8


def test_route_backward_leaves_out_what_was_not_chosen():
    l = torch.zeros(1, 8, device=DEV)
    l[0, 5] = -math.inf
    ids = torch.tensor([[2, -1, 5, 99]], dtype=torch.int32, device=DEV)
    dw = torch.tensor([[1.0, math.nan, math.nan, math.nan]], device=DEV)
    none = torch.full_like(l, -math.inf)
    for scoring in ("sigmoid", "softmax"):
        for renormalize in (True, False):  # a row of nothing but unavailable experts
            d = F.moe_route_topk_backward(none, ids, dw, scoring=scoring, renormalize=renormalize)
            assert torch.equal(d, torch.zeros_like(d))
        d = F.moe_route_topk_backward(l, ids, dw, scoring=scoring, renormalize=True)
        assert torch.equal(d, torch.zeros_like(d))  # a single weight of 1 whatever its logit
        d = F.moe_route_topk_backward(l, ids, dw, scoring=scoring, renormalize=False)
        assert d.isfinite().all() and d[0, 2] > 0 and d[0, 5] == 0


# ------------------------------------------------------------------ combine

def pairs(seed, T, k, E, M):
    """ids, slots [T, k]: some pairs without a row (id or slot outside), no row named twice."""
    g = rng(3, seed)
    rows = g.permutation(E * M)[:T * k]
    rows = np.concatenate([rows, np.full(T * k - rows.size, -1)])
    ids, slots = rows // M, rows % M
    none = g.random(T * k)
    ids = np.where((rows < 0) | (none < 0.06), g.choice([-1, E, E + 7], T * k), ids)
    slots = np.where((none > 0.94), g.choice([-1, M, M + 3], T * k), slots)
    return ids.reshape(T, k).astype(np.int32), slots.reshape(T, k).astype(np.int32)


def poison_rows(y, ids, slots):
    """NaN in the rows that no pair names."""
    E, M, N = y.shape
    ok = (ids >= 0) & (ids < E) & (slots >= 0) & (slots < M)
    used = np.zeros((E, M), bool)
    used[ids[ok], slots[ok]] = True
    y = y.copy()
    y[~used] = np.nan
    return y, used, ok


COMBINES = [(1, 1, 1, 1, 8), (3, 2, 4, 8, 64), (65, 8, 9, 80, 2048), (7, 9, 33, 4, 2056), (2, 64, 64, 8, 1032),
            (5, 6, 3, 40, 7168)]


@pytest.mark.parametrize("T,k,E,M,N", COMBINES)
@pytest.mark.parametrize("weighted,based", [(True, True), (False, False), (True, False)])
def test_combine(T, k, E, M, N, weighted, based):
    g = rng(4, T, N)
    ids, slots = pairs(T + k, T, k, E, M)
    y, y64 = bf(poison_rows(g.normal(size=(E, M, N)), ids, slots)[0])
    w, w64 = f32(g.random((T, k))) if weighted else (None, None)
    b, b64 = bf(g.normal(size=(T, N))) if based else (None, None)
    out = nans(T, N + 16)
    got = F.moe_combine(y, torch.from_numpy(ids).to(DEV), torch.from_numpy(slots).to(DEV), w,
                        base=None if b is None else strided(b, 8), out=out[:, :N])
    assert got.data_ptr() == out.data_ptr() and out[:, N:].isnan().all()
    ref, mag = R.combine(y64, ids, slots, w64, b64)
    close(got, ref, R.BF16_U * np.abs(ref) + (k + 1) * R.F32_U * mag)


@pytest.mark.parametrize("T,k,E,M,N", COMBINES)
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("quantize", [False, True])
def test_combine_backward(T, k, E, M, N, weighted, quantize):
    if quantize:
        N = -(-N // 128) * 128
    g = rng(5, T, N)
    ids, slots = pairs(T + k, T, k, E, M)
    yn, used, ok = poison_rows(g.normal(size=(E, M, N)), ids, slots)
    y, y64 = bf(yn)
    w, w64 = f32(g.normal(size=(T, k))) if weighted else (None, np.ones((T, k)))
    d, d64 = bf(g.normal(size=(T, N)) * np.exp(g.normal(size=(T, 1)) * 4))
    args = (strided(d, 16), y, torch.from_numpy(ids).to(DEV), torch.from_numpy(slots).to(DEV), w)
    if quantize:
        q = torch.full((E, M, N), 0xAB, dtype=torch.uint8, device=DEV)
        sf = torch.full((E, (N // 128 + 3) // 4, M), -7, dtype=torch.int32, device=DEV)
        _, _, dw = F.moe_combine_backward(*args, quantize=True, q=q, sf=sf)
        qh, sfh = q.cpu().numpy(), sf.cpu().numpy()
        assert (qh[~used] == 0xAB).all() and (sfh.transpose(0, 2, 1)[~used] == -7).all()
        for t, j in np.argwhere(ok):
            e, s = ids[t, j], slots[t, j]
            v = (w64[t, j] * d64[t])[None]
            R.check_quantized(v, qh[e, s][None], sfh[e, :, s:s + 1].copy(), 2 * R.F32_U * np.abs(v))
    else:
        dy = nans(E, M, N)
        _, dw = F.moe_combine_backward(*args, d_y=dy)
        h = host(dy)
        assert np.isnan(h[~used]).all()
        ref = np.zeros((E, M, N))
        for t, j in np.argwhere(ok):
            ref[ids[t, j], slots[t, j]] = w64[t, j] * d64[t]
        close(h[used], ref[used], (R.BF16_U + 2 * R.F32_U) * np.abs(ref[used]))
    if not weighted:
        assert dw is None
        return
    for t in range(T):
        for j in range(k):
            if ok[t, j]:
                terms = d64[t] * y64[ids[t, j], slots[t, j]]
                # products are exact in fp32 before their sum: N additions at the most
                assert abs(float(dw[t, j]) - terms.sum()) <= N * R.F32_U * np.abs(terms).sum()
            else:
                assert float(dw[t, j]) == 0.0


def test_combine_backward_is_the_derivative():
    # <d_out, combine> is linear in y and in weights: its differences are exact
    T, k, E, M, N = 4, 3, 5, 4, 64
    g = rng(6)
    ids, slots = pairs(2, T, k, E, M)
    y, y64 = bf(np.nan_to_num(g.normal(size=(E, M, N))))
    w, w64 = f32(g.normal(size=(T, k)))
    d, d64 = bf(g.normal(size=(T, N)))
    it, st = torch.from_numpy(ids).to(DEV), torch.from_numpy(slots).to(DEV)
    dy, dw = F.moe_combine_backward(d, y, it, st, w, d_y=torch.zeros_like(y))

    def value(yv, wv):
        return (R.combine(yv, ids, slots, wv, None)[0] * d64).sum()
    dirs = g.normal(size=y64.shape), g.normal(size=w64.shape)
    by_y = value(y64 + dirs[0], w64) - value(y64, w64)
    assert abs((host(dy) * dirs[0]).sum() - by_y) <= R.BF16_U * (np.abs(host(dy) * dirs[0])).sum() + 1e-9
    by_w = value(y64, w64 + dirs[1]) - value(y64, w64)
    assert abs((host(dw) * dirs[1]).sum() - by_w) <= 1e-5 * np.abs(host(dw) * dirs[1]).sum() + 1e-9


def test_combine_of_an_empty_layout():
    ids = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    y = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    base = torch.randn(3, 64, device=DEV).to(BF)
    assert torch.equal(F.moe_combine(y, ids, ids, base=base), base)
    w = torch.ones(3, 2, device=DEV)
    _, dw = F.moe_combine_backward(base, y, ids, ids, w)
    assert torch.equal(dw, torch.zeros_like(dw))
    assert F.moe_combine(y, ids[:0], ids[:0]).shape == (0, 64)


def test_combine_past_32_bits():
    E, M, N = 2, 70000, 16384  # 4.6 GB of rows
    y = torch.empty(E, M, N, dtype=BF, device=DEV)
    rows = torch.randn(2, N, device=DEV).to(BF)
    y[1, M - 1], y[0, 0] = rows[0], rows[1]
    ids = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    slots = torch.tensor([[M - 1, 0]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[1.0, 2.0]], device=DEV)
    out = F.moe_combine(y, ids, slots, w)
    assert torch.equal(out[0], (rows[0].float() + 2 * rows[1].float()).to(BF))
    dy, dw = F.moe_combine_backward(out, y, ids, slots, w, d_y=y.clone())
    assert torch.equal(dy[1, M - 1], out[0]) and torch.equal(dy[0, 0], (2 * out[0].float()).to(BF))


# ------------------------------------------------------------------ residual norms

NORMS = [(1, 8), (2, 128), (5, 520), (300, 256), (3, 2048), (2, 7168), (65, 1544), (2, 8200), (2, 16384)]
PARTS = [("none", False), ("channel", True), ("full", True), ("channel", False), ("before", False)]


def norm_inputs(seed, T, N, gate, post, res):
    g = rng(7, seed, N)
    make = f32 if res == torch.float32 else bf
    a = {"x": make(g.normal(size=(T, N)) * 2), "w_pre": bf(1 + 0.2 * g.normal(size=N)), "y": (None, None),
         "w_post": (None, None), "gate": (None, None)}
    if gate != "before":
        yv = g.normal(size=(T, N)) * np.exp(g.normal(size=(T, 1)) * 3)
        if T > 1:
            yv[0] = 0  # a branch of zeros: its norm divides by sqrt(eps)
        a["y"] = bf(yv)
        if post:
            a["w_post"] = bf(1 + 0.2 * g.normal(size=N))
        if gate in ("channel", "full"):
            a["gate"] = bf(g.normal(size=N if gate == "channel" else (T, N)))
    return g, {n: v[0] for n, v in a.items()}, {n: v[1] for n, v in a.items()}


def rel_of_norm(N):
    """Relative error of an fp32 1 / sqrt(mean square): half of N + 4 roundings, and two of rsqrt."""
    return (N / 2 + 6) * R.F32_U


@pytest.mark.parametrize("T,N", NORMS)
@pytest.mark.parametrize("gate,post", PARTS)
@pytest.mark.parametrize("res", [BF, torch.float32])
def test_norm(T, N, gate, post, res):
    g, a, v = norm_inputs(1, T, N, gate, post, res)
    scale, offset = (0.75, 1.0) if T % 2 else (1.0, 0.0)
    href, zref = R.norm(v["x"], v["w_pre"], v["y"], v["w_post"], v["gate"], scale, 1e-5, offset)
    out = "both" if N % 128 == 0 else "bf16"
    x = strided(a["x"], 8)
    h, z, q, sf = F.residual_rms_norm(x, a["w_pre"], y=None if a["y"] is None else strided(a["y"], 16), w_post=a["w_post"],
                                      gate=a["gate"] if a["gate"] is None or a["gate"].dim() == 1 else strided(a["gate"], 8),
                                      residual_scale=scale, eps=1e-5, weight_offset=offset, out=out,
                                      z=nans(T, N + 8)[:, :N])
    # magnitudes of the terms of h: what their rounding is relative to
    mag = np.abs(scale * v["x"]) + np.abs(href - scale * v["x"])
    herr = (rel_of_norm(N) + 6 * R.F32_U) * mag
    if a["y"] is None and scale == 1.0:
        assert h is x
    else:
        close(h, href, herr + (R.BF16_U * np.abs(href) if res == BF else 0), "h")
    r = R.rms(href, 1e-5)
    zerr = (herr + (rel_of_norm(N) + 4 * R.F32_U + herr.max(-1, keepdims=True) * r) * np.abs(href)) * r * np.abs(
        v["w_pre"] + offset)
    close(z, zref, zerr + R.BF16_U * np.abs(zref), "z")
    if out == "both":
        R.check_quantized(zref, q.cpu().numpy(), sf.cpu().numpy(), zerr)


def test_norm_codes_are_the_quantization_of_the_norm():
    # weights and scales of powers of two, so that z is exact in bf16 and the two ways have the same input
    T, N = 9, 1024
    x = torch.sign(torch.randn(T, N, device=DEV)).to(BF) * torch.exp2(torch.arange(T, device=DEV).float() - 4).unsqueeze(1).to(BF)
    w = torch.exp2(torch.randint(-3, 4, (N,), device=DEV).float()).to(BF)
    _, z, q, sf = F.residual_rms_norm(x, w, eps=0.0, out="both")
    q2, sf2 = F.fp8_quant_group_pack(z)
    assert torch.equal(q, q2) and torch.equal(sf[:, :T], sf2[:, :T])


@pytest.mark.parametrize("T,N", NORMS)
@pytest.mark.parametrize("gate,post", PARTS)
@pytest.mark.parametrize("res", [BF, torch.float32])
def test_norm_backward(T, N, gate, post, res):
    g, a, v = norm_inputs(2, T, N, gate, post, res)
    scale, offset, eps = (0.75, 1.0, 1e-5) if T % 2 else (1.0, 0.0, 1e-3)
    dz, dz64 = bf(g.normal(size=(T, N)))
    dh, dh64 = (f32 if res == torch.float32 else bf)(g.normal(size=(T, N)))
    with_dh = gate != "none"
    got = F.residual_rms_norm_backward(strided(dz, 8), strided(a["x"], 8), a["w_pre"], d_h=strided(dh, 24) if with_dh else None,
                                       y=a["y"], w_post=a["w_post"], gate=a["gate"], residual_scale=scale, eps=eps,
                                       weight_offset=offset, d_x=nans(T, N + 8, dtype=res)[:, :N])
    # the formulas by automatic differentiation in 64 bits; "x" is h here
    leaf = {n: torch.from_numpy(t).requires_grad_(True) for n, t in v.items() if t is not None}

    def normed(t, w):
        return t * torch.rsqrt((t * t).mean(-1, keepdim=True) + eps) * (w + offset)
    h = leaf["x"]
    dh_t, dw_pre = torch.autograd.grad((normed(h, leaf["w_pre"]) * torch.from_numpy(dz64)).sum(), [h, leaf["w_pre"]])
    if with_dh:
        dh_t = dh_t + torch.from_numpy(dh64)
    ref = {"x": scale * dh_t, "w_pre": dw_pre}
    if "y" in leaf:
        b = leaf["y"] if "w_post" not in leaf else normed(leaf["y"], leaf["w_post"])
        b = b if "gate" not in leaf else b * leaf["gate"]
        names = [n for n in ("y", "w_post", "gate") if n in leaf]
        ref.update(zip(names, torch.autograd.grad((b * dh_t).sum(), [leaf[n] for n in names])))
    # errors: every term of a row's gradient is within (rel_of_norm + 8 roundings) and each of the two
    # inner means adds N roundings of a mean of magnitudes; the rows' largest magnitudes bound them
    rel = 2 * rel_of_norm(N) + (N + 32) * R.F32_U
    rh = R.rms(v["x"], eps)
    wp = np.abs(v["w_pre"] + offset)
    top = lambda m: m.max(-1, keepdims=True)  # noqa: E731
    dz_mag = top(np.abs(dz64) * wp)
    dh_mag = rh * dz_mag * (1 + top(np.abs(v["x"])) * rh) + (top(np.abs(dh64)) if with_dh else 0)
    xerr = rel * scale * dh_mag * np.ones((1, N))
    xr = ref["x"].numpy()
    close(got[0], xr, xerr + (R.BF16_U * np.abs(xr) if res == BF else 0), "d_x")
    hh_mag = np.abs(v["x"]) * rh
    close(got[2], ref["w_pre"].numpy(), (rel + T * R.F32_U) * (np.abs(dz64) * hh_mag).sum(0), "d_w_pre")
    if "y" not in leaf:
        assert got[1] is None and got[3] is None and got[4] is None
        return
    gt = np.abs(v["gate"]) if v["gate"] is not None else np.ones((1, N))
    yh = np.abs(v["y"])
    db_mag = dh_mag * top(gt * np.ones((T, N)))
    y_mag = db_mag
    if post:
        ry = R.rms(v["y"], eps)
        yh = yh * ry
        wpo = np.abs(v["w_post"] + offset)
        y_mag = ry * db_mag * wpo.max() * (1 + top(yh))
        close(got[3], ref["w_post"].numpy(), (2 * rel + T * R.F32_U) * (db_mag * yh).sum(0) + 1e-30, "d_w_post")
        b_mag = yh * wpo
    else:
        assert got[3] is None
        b_mag = yh
    yr = ref["y"].numpy()
    close(got[1], yr, R.BF16_U * np.abs(yr) + 2 * rel * y_mag * np.ones((1, N)), "d_y")
    if v["gate"] is None:
        assert got[4] is None
    elif v["gate"].ndim == 1:
        assert got[4].dtype == torch.float32
        close(got[4], ref["gate"].numpy(), (2 * rel + T * R.F32_U) * (dh_mag * b_mag).sum(0) + 1e-30, "d_gate")
    else:
        assert got[4].dtype == BF
        gr = ref["gate"].numpy()
        close(got[4], gr, R.BF16_U * np.abs(gr) + 2 * rel * dh_mag * b_mag + 1e-30, "d_gate")


def test_norm_backward_against_differences():
    T, N, eps, step = 3, 64, 1e-4, 1e-5
    g, a, v = norm_inputs(3, T, N, "channel", True, torch.float32)
    dz, dz64 = bf(g.normal(size=(T, N)))
    # h as the forward has it, from x = v["x"] in 64 bits; then fp32 for the call
    h64, _ = R.norm(v["x"], v["w_pre"], v["y"], v["w_post"], v["gate"], 0.5, eps)
    got = F.residual_rms_norm_backward(dz, f32(h64)[0], a["w_pre"], y=a["y"], w_post=a["w_post"], gate=a["gate"],
                                       residual_scale=0.5, eps=eps)

    def value(**over):
        u = {**v, **over}
        return (R.norm(u["x"], u["w_pre"], u["y"], u["w_post"], u["gate"], 0.5, eps)[1] * dz64).sum()
    for name, grad in zip(("x", "y", "w_pre", "w_post", "gate"), got):
        d = g.normal(size=v[name].shape)
        if name == "y":
            d[0] = 0  # (the row of zeros is at the norm's kink: its step would have to be far below sqrt(eps))
        diff = (value(**{name: v[name] + step * d}) - value(**{name: v[name] - step * d})) / (2 * step)
        terms = host(grad) * d
        # bf16 gradients (d_y): 2^-8 of each term; differences: step^2
        assert abs(terms.sum() - diff) <= 2 ** -8 * np.abs(terms).sum() + 1e-5, name


def test_norm_of_nothing_and_of_zeros():
    w = torch.ones(256, dtype=BF, device=DEV)
    h, z, q, sf = F.residual_rms_norm(torch.zeros(2, 256, dtype=BF, device=DEV), w, residual_scale=3.0, out="both")
    assert not h.any() and not z.any() and not q.any()
    assert (sf[:, :2] == 85 | 85 << 8).all()  # the exponent floor of two groups
    e = torch.empty(0, 256, dtype=BF, device=DEV)
    h, z, q, sf = F.residual_rms_norm(e, w, y=e, w_post=w, gate=w, out="both")
    assert h.shape == z.shape == q.shape == (0, 256)
    d = nans(256, dtype=torch.float32)
    got = F.residual_rms_norm_backward(e, e, w, y=e, w_post=w, gate=w, d_w_pre=d, d_w_post=d.clone(), d_gate=d.clone())
    for t in got[2:]:
        assert torch.equal(t, torch.zeros_like(t))


def test_norm_keeps_bad_rows_to_themselves():
    x = torch.randn(4, 512, device=DEV).to(BF)
    w = torch.ones(512, dtype=BF, device=DEV)
    _, clean, _, _ = F.residual_rms_norm(x, w, y=x, w_post=w)
    x2 = x.clone()
    x2[1, 3], x2[2, 7] = math.nan, math.inf
    _, z, _, _ = F.residual_rms_norm(x2, w, y=x2, w_post=w)
    assert torch.equal(z[[0, 3]], clean[[0, 3]]) and z[1].isnan().all() and z[2, 7].isnan()


def test_norm_past_32_bits():
    T, N = 140000, 16384  # rows of 4.6 GB
    x = torch.zeros(T, N, dtype=BF, device=DEV)
    x[-1] = torch.randn(N, device=DEV).to(BF)
    w = torch.ones(N, dtype=BF, device=DEV)
    h, z, _, _ = F.residual_rms_norm(x, w, y=x, w_post=w, gate=w)
    h1, z1, _, _ = F.residual_rms_norm(x[-1:], w, y=x[-1:], w_post=w, gate=w)
    assert torch.equal(h[-1:], h1) and torch.equal(z[-1:], z1) and not z[:-1].any()


# ------------------------------------------------------------------ 8-bit checkpoint

CHECKPOINTS = [([1], 1, 128), ([0, 5, 8, 3, 20, -4], 8, 256), ([7, 0, 0, 33], 33, 640), ([256] * 3, 256, 2048),
               (list(range(70)), 64, 128), ([0] * 299 + [2], 3, 384), ([0, 0, 0], 4, 128)]


@pytest.mark.parametrize("counts,M,H", CHECKPOINTS, ids=lambda v: str(v)[:12])
def test_checkpoint(counts, M, H):
    E = len(counts)
    g = rng(8, E, H)
    xn = g.normal(size=(E, M, 2 * H)) * np.exp(g.normal(size=(E, M, 1)) * 2)
    valid = np.arange(M) < np.clip(counts, 0, M)[:, None]
    xn[~valid] = np.nan
    x, x64 = bf(xn)
    m = torch.tensor(counts, dtype=torch.int32, device=DEV)
    W = (H // 128 + 3) // 4
    bufs = [torch.full((E, M, H), 0xAB, dtype=torch.uint8, device=DEV),
            torch.full((E, W, M), -7, dtype=torch.int32, device=DEV),
            torch.full((E, M, 2 * H), 0xAB, dtype=torch.uint8, device=DEV),
            torch.full((E, 2 * W, M), -7, dtype=torch.int32, device=DEV)]
    q, sf, cq, csf = F.silu_mul_quant_group_pack_checkpoint(x, m, *bufs)
    q2, sf2 = F.silu_mul_quant_group_pack(x, m, q=torch.full_like(q, 0xAB), sf=torch.full_like(sf, -7))
    assert torch.equal(q, q2) and torch.equal(sf, sf2)  # the same bits, padded rows untouched too
    v = torch.from_numpy(valid).to(DEV)
    assert (cq[~v] == 0xAB).all() and (csf.transpose(1, 2)[~v] == -7).all()
    for half in (0, 1):  # value for value the per-token quantization of each half
        part = x[..., half * H:(half + 1) * H].reshape(E * M, H).contiguous()
        rq, rsf = F.fp8_quant_group_pack(part)
        assert torch.equal(cq[..., half * H:(half + 1) * H][v], rq.view(E, M, H)[v])
        rows = csf[:, half * W:(half + 1) * W].transpose(1, 2)[v]
        assert torch.equal(rows, rsf[:, :E * M].t().reshape(E, M, W)[v])


def test_checkpoint_of_every_gate():
    # every finite bf16 pattern as a gate: the same codes as the forward without a checkpoint
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    gate = torch.from_numpy(bits.view(np.int16)).view(BF).to(DEV).reshape(1, -1, 128)
    x = torch.cat([gate, torch.ones_like(gate)], -1).contiguous()
    m = torch.tensor([x.shape[1]], dtype=torch.int32, device=DEV)
    q, sf, _, _ = F.silu_mul_quant_group_pack_checkpoint(x, m)
    q2, sf2 = F.silu_mul_quant_group_pack(x, m)
    assert torch.equal(q, q2) and torch.equal(sf, sf2)


def test_values_that_are_not_finite_become_nan_codes():
    x = torch.randn(1, 3, 512, device=DEV).to(BF)
    x[0, 1, 5], x[0, 1, 300] = math.nan, math.inf
    m = torch.tensor([3], dtype=torch.int32, device=DEV)
    q, _, cq, _ = F.silu_mul_quant_group_pack_checkpoint(x, m)
    nan = lambda c: c.view(torch.float8_e4m3fn).float().isnan().nonzero().tolist()  # noqa: E731
    assert nan(cq) == [[0, 1, 5], [0, 1, 300]]
    assert [0, 1, 5] in nan(q) and [0, 1, 44] in nan(q)
    w = torch.ones(256, dtype=BF, device=DEV)
    _, _, q, _ = F.residual_rms_norm(x[0, :, :256].contiguous(), w, out="fp8")
    assert nan(q)[0][0] == 1 and nan(q)[-1][0] == 1  # row 1 and no other
    ids, slots = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    q, _, _ = F.moe_combine_backward(x[0, 1:2, :256].contiguous(), x[:, :1, :256].contiguous(), ids, slots, quantize=True)
    assert nan(q) == [[0, 0, 5]]


def checkpoint_of(x, m):
    _, _, cq, csf = F.silu_mul_quant_group_pack_checkpoint(x, m)
    E, M, H2 = x.shape
    H = H2 // 2
    W = (H // 128 + 3) // 4
    c, s = cq.cpu().numpy(), csf.cpu().numpy()
    val = np.zeros((E, M, H2))
    for e in range(E):
        for half in (0, 1):
            b = np.ascontiguousarray(s[e, half * W:(half + 1) * W]).view(np.uint32)
            b = np.stack([(b >> (8 * i)) & 0xFF for i in range(4)], -1).transpose(1, 0, 2).reshape(M, -1)[:, :H // 128]
            val[e, :, half * H:(half + 1) * H] = R.e4m3_decode(c[e, :, half * H:(half + 1) * H]) * np.repeat(
                2.0 ** (b.astype(np.int64) - 127.0), 128, 1)
    return cq, csf, val


@pytest.mark.parametrize("counts,M,H", CHECKPOINTS, ids=lambda v: str(v)[:12])
@pytest.mark.parametrize("quantize", [False, True])
def test_checkpoint_backward(counts, M, H, quantize):
    E = len(counts)
    g = rng(9, E, H)
    xn = g.normal(size=(E, M, 2 * H)) * 3
    xn[..., 0] = np.where(g.random((E, M)) < 0.5, 150.0, -150.0)  # gates where sigmoid or its rest underflow
    xn[..., 1] = 0
    x, _ = bf(xn)
    full = torch.full((E,), M, dtype=torch.int32, device=DEV)
    cq, csf, val = checkpoint_of(x, full)
    n = np.clip(counts, 0, M)
    valid = np.arange(M) < n[:, None]
    d, d64 = bf(np.where(valid[..., None], g.normal(size=(E, M, H)), np.nan))
    m = torch.tensor(counts, dtype=torch.int32, device=DEV)
    gate, up = val[..., :H], val[..., H:]
    s, rest = R.sigmoid(gate), R.sigmoid(-gate)
    ref = np.concatenate([d64 * up * s * (1 + gate * rest), d64 * gate * s], -1)
    # 1 + gate * (1 - s) is a difference for negative gates: relative to 1 + |gate| (1 - s)
    mag = np.concatenate([np.abs(d64 * up) * s * (1 + np.abs(gate) * rest), np.abs(d64 * gate) * s], -1)
    W2 = (2 * H // 128 + 3) // 4
    if quantize:
        q = torch.full((E, M, 2 * H), 0xAB, dtype=torch.uint8, device=DEV)
        sf = torch.full((E, W2, M), -7, dtype=torch.int32, device=DEV)
        F.silu_mul_backward_from_checkpoint(d, m, cq, csf, quantize=True, q=q, sf=sf)
        qh, sfh = q.cpu().numpy(), sf.cpu().numpy()
        assert (qh[~valid] == 0xAB).all() and (sfh.transpose(0, 2, 1)[~valid] == -7).all()
        for e in range(E):
            if n[e]:
                R.check_quantized(ref[e, :n[e]], qh[e, :n[e]], sfh[e, :, :n[e]].copy(), 16 * R.F32_U * mag[e, :n[e]] + 1e-36)
    else:
        dx = nans(E, M, 2 * H)
        F.silu_mul_backward_from_checkpoint(d, m, cq, csf, d_x=dx)
        h = host(dx)
        assert np.isnan(h[~valid]).all()
        # exp of a rounded argument, reciprocal, four products: 16 roundings; exp underflows below 2^-126
        close(h[valid], ref[valid], R.BF16_U * np.abs(ref[valid]) + 16 * R.F32_U * mag[valid] + 1e-36)


def test_checkpoint_backward_is_the_derivative_at_the_checkpoint():
    E, M, H, step = 1, 2, 128, 1e-6
    g = rng(10)
    x, _ = bf(g.normal(size=(E, M, 2 * H)))
    m = torch.tensor([M], dtype=torch.int32, device=DEV)
    cq, csf, val = checkpoint_of(x, m)
    d, d64 = bf(g.normal(size=(E, M, H)))
    dx = host(F.silu_mul_backward_from_checkpoint(d, m, cq, csf))
    dirs = g.normal(size=val.shape)

    def value(v):
        return (v[..., :H] * R.sigmoid(v[..., :H]) * v[..., H:] * d64).sum()
    diff = (value(val + step * dirs) - value(val - step * dirs)) / (2 * step)
    assert abs((dx * dirs).sum() - diff) <= R.BF16_U * np.abs(dx * dirs).sum() + 1e-6


def test_checkpoint_past_32_bits():
    E, M, H = 2, 140000, 8192  # 2 * 140000 * 16384 codes
    x = torch.zeros(E, M, 2 * H, dtype=BF, device=DEV)
    x[1, M - 1] = torch.randn(2 * H, device=DEV).to(BF)
    m = torch.full((E,), M, dtype=torch.int32, device=DEV)
    q, sf, cq, csf = F.silu_mul_quant_group_pack_checkpoint(x, m)
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    last = F.silu_mul_quant_group_pack_checkpoint(x[1:, M - 1:].contiguous(), one)
    for t, t1 in zip((q, cq), (last[0], last[2])):
        assert torch.equal(t[1, M - 1], t1[0, 0]) and not t[:, :M - 1].any()
    assert torch.equal(csf[1, :, M - 1], last[3][0, :, 0]) and torch.equal(sf[1, :, M - 1], last[1][0, :, 0])
    del x, q
    d = torch.ones(E, M, H, dtype=BF, device=DEV)
    dx = F.silu_mul_backward_from_checkpoint(d, m, cq, csf)
    dx1 = F.silu_mul_backward_from_checkpoint(d[:1, :1].contiguous(), one, last[2], last[3])
    assert torch.equal(dx[1, M - 1], dx1[0, 0])


# ------------------------------------------------------------------ streams, graphs, repeatability

def chain(s):
    """All the operators once, on tensors of the state s; every output."""
    ids, w = F.moe_route_topk(s["logits"], 4, bias=s["bias"], groups=4, topk_groups=2, group_top=2, scoring="sigmoid")
    q, sf, m, slots = F.fp8_quant_group_pack_to_experts(s["x"], ids, 16, 32, q=s["q"], sf=s["sf"])
    out = F.moe_combine(s["y"], ids, slots, w, base=s["x"])
    dy, dw = F.moe_combine_backward(s["x"], s["y"], ids, slots, w, d_y=s["dy"])
    dl = F.moe_route_topk_backward(s["logits"], ids, dw, scoring="sigmoid")
    h, z, qz, sfz = F.residual_rms_norm(s["x"], s["w"], y=out, w_post=s["w"], gate=s["w"], out="both")
    grads = F.residual_rms_norm_backward(z, h, s["w"], d_h=h, y=out, w_post=s["w"], gate=s["w"])
    cks = F.silu_mul_quant_group_pack_checkpoint(s["y"], m, *s["ck"])
    dx = F.silu_mul_backward_from_checkpoint(s["dy_half"], m, cks[2], cks[3], d_x=s["dx"])
    return [ids, w, out, dy, dw, dl, h, z, qz, *grads, *cks, dx]


def chain_state(seed):
    torch.manual_seed(seed)
    T, N, E, M = 48, 512, 16, 32
    z = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    r = lambda *s: torch.randn(*s, device=DEV).to(BF)  # noqa: E731
    return dict(logits=torch.randn(T, E, device=DEV), bias=torch.rand(E, device=DEV), x=r(T, N), y=r(E, M, N),
                q=z(E, M, N, dtype=torch.uint8), sf=z(E, 1, M, dtype=torch.int32), dy=z(E, M, N), w=r(N),
                ck=[z(E, M, N // 2, dtype=torch.uint8), z(E, 1, M, dtype=torch.int32), z(E, M, N, dtype=torch.uint8),
                    z(E, 2, M, dtype=torch.int32)], dy_half=r(E, M, N // 2), dx=z(E, M, N))


def bits(outs):
    return [t.contiguous().view(torch.uint8).clone() for t in outs]


def test_on_another_stream_and_again():
    s = chain_state(1)
    torch.cuda.synchronize()
    first = bits(chain(s))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        second = bits(chain(s))
    torch.cuda.current_stream().wait_stream(other)
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    # and with the stream as an argument
    ids, w = F.moe_route_topk(s["logits"], 4, scoring="softmax", stream=other)
    ids3, w3 = F.moe_route_topk(s["logits"], 4, scoring="softmax", stream=other.cuda_stream)  # or its handle
    other.synchronize()
    ids2, w2 = F.moe_route_topk(s["logits"], 4, scoring="softmax")
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    assert torch.equal(ids3, ids2) and torch.equal(w3, w2)


def test_graph_replays():
    s = chain_state(2)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = bits(chain(s))  # also grows the stream's workspace, which a capture may not
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs = chain(s)
    torch.cuda.synchronize()
    for i in range(4):
        for t in outs:
            if i % 2:
                t.view(torch.uint8).fill_(0x11)
        for name in ("q", "dy", "dx"):
            s[name].zero_()
        for t in s["ck"] + [s["sf"]]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = bits(outs)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        eager = chain_state(3)
        with torch.cuda.stream(stream):
            chain(eager)  # eager work on the same workspace between the replays
        torch.cuda.synchronize()


def test_other_device_tensors_are_refused():
    with pytest.raises(ValueError, match="device tensor"):
        F.moe_route_topk(torch.zeros(2, 8, device=DEV), 2, bias=torch.zeros(8))
    with pytest.raises(ValueError, match="device tensor"):
        F.moe_route_topk(torch.zeros(2, 8, device=DEV), 2, weights=torch.zeros(2, 2))
