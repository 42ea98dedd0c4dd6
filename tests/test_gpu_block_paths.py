"""The routing's vector loads and stores, and the loops over several rows or units of one
workgroup, which long calls take: against references in 64 bits, and bit for bit against the
same rows in other layouts and in calls so short that no loop runs twice.

Bounds count roundings: u = 2^-24 for every fp32 operation, and sums by the depth of their
tree (a thread's own terms one after the other, then lanes and wavefronts pairwise).  Where an
output is rounded to bf16 it has to lie between the roundings of the two ends of that bound."""
import numpy as np
import pytest
import torch

import block_reference as R
import block_scaled_fp8_token_amd as F
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = R.F32_U


def gen(*seed):
    return np.random.default_rng([30, *seed])


# ------------------------------------------------------------------ routing

CONTIGUOUS = [  # T, E, topk, groups, topk_groups, group_top, scoring, bias: rows of whole 16-byte words
    (5, 64, 8, 1, 1, 1, "softmax", False),
    (7, 128, 6, 1, 1, 1, "softmax", True),
    (66, 256, 8, 8, 4, 2, "sigmoid", True),
    (33, 256, 8, 4, 2, 1, "softmax", False),
    (13, 512, 8, 1, 1, 1, "sigmoid", False),
    (9, 512, 7, 16, 4, 2, "sigmoid", True),
    (6, 160, 6, 1, 1, 1, "softmax", False),
    (10, 256, 9, 8, 4, 2, "sigmoid", True),
    (3, 1024, 16, 1, 1, 1, "softmax", False),
    (1, 256, 8, 8, 4, 2, "sigmoid", True),
]


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("i", range(len(CONTIGUOUS)))
def test_route_of_contiguous_rows(i, masked, dtype):
    T, E, k, G, kg, top, scoring, bias = CONTIGUOUS[i]
    g = gen(1, i, int(masked))
    l = np.clip(np.round(g.normal(size=(T, E)) * 24) / 16, -7, 7)  # exact in bf16, with ties
    if masked:
        l[g.random((T, E)) < 0.3] = -np.inf
        l[g.random((T, E)) < 0.05] = np.nan
        l[0] = -np.inf
        if T > 2:
            l[1, 1:], l[1, 0] = np.nan, 0.5
            l[2, E // 2] = np.inf
    b = g.integers(-4, 5, E) / 8.0 if bias else None
    bt = None if b is None else torch.from_numpy(b).float().to(DEV)
    lt = torch.from_numpy(l).to(dtype).to(DEV)
    wide = torch.full((T, E + 24), float("nan"), dtype=dtype, device=DEV)
    wide[:, 8:8 + E] = lt  # aligned rows with a stride
    odd = torch.full((T, E + 3), float("nan"), dtype=dtype, device=DEV)
    odd[:, 1:1 + E] = lt  # rows that no wide load can take
    for renormalize in (True, False):
        opts = dict(groups=G, topk_groups=kg, group_top=top, scoring=scoring, renormalize=renormalize, scale=1.5)
        ids, w, gap = R.route(l, k, bias=b, **opts)
        assert gap > 1e-6
        got_ids, got_w = F.moe_route_topk(lt, k, bias=bt, **opts)
        assert np.array_equal(got_ids.cpu().numpy(), ids)
        got = got_w.double().cpu().numpy()
        assert (np.abs(got - w) <= (E + k + 16) * U * np.abs(w) + 1e-37).all()  # sums of E and k, a few roundings
        for other in (wide[:, 8:8 + E], odd[:, 1:1 + E]):
            o_ids, o_w = F.moe_route_topk(other, k, bias=bt, **opts)
            assert torch.equal(o_ids, got_ids) and torch.equal(o_w, got_w)
        if bias:  # a bias that no wide load can take
            o_ids, o_w = F.moe_route_topk(lt, k, bias=torch.cat([bt[:1], bt])[1:], **opts)
            assert torch.equal(o_ids, got_ids) and torch.equal(o_w, got_w)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("scoring,renormalize", [("softmax", False), ("softmax", True), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k", [(6, 128, 8), (7, 160, 6), (9, 256, 8), (5, 512, 10), (3, 1024, 64), (1, 256, 1)])
def test_route_backward_of_contiguous_rows(T, E, k, scoring, renormalize, dtype):
    g = gen(2, T, E)
    l = torch.from_numpy(np.clip(g.normal(size=(T, E)) * 1.5, -6, 6)).to(dtype)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    ids[:, 0] = g.choice([0, E - 1], T)  # the ends of the lanes' pieces
    for t in range(T):
        ids[t, 1:] = [e for e in g.permutation(E) if e != ids[t, 0]][:k - 1]
    dw = torch.from_numpy(g.normal(size=(T, k)).astype(np.float32))
    opts = dict(scoring=scoring, renormalize=renormalize, scale=1.75)
    args = torch.from_numpy(ids).int().to(DEV), dw.to(DEV)
    lt = l.to(DEV)
    got = F.moe_route_topk_backward(lt, *args, d_logits=torch.full_like(lt, float("nan")), **opts)
    # the formula, by automatic differentiation in 64 bits
    ld = l.double().requires_grad_(True)
    s = torch.sigmoid(ld) if scoring == "sigmoid" else torch.softmax(ld, 1)
    w = s.gather(1, torch.from_numpy(ids))
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    ref = torch.autograd.grad((w * dw.double()).sum() * 1.75, ld)[0].numpy()
    # a product with a difference of dw and a mean of dw, of the magnitude 2 c max|dw| max(w)
    scale = 2 * 1.75 * float(dw.abs().max()) * w.detach().numpy().max(1, keepdims=True)
    bound = (E + 2 * k + 24) * U * scale + (R.BF16_U * np.abs(ref) if dtype == BF else 0)
    assert (np.abs(got.double().cpu().numpy() - ref) <= bound).all()
    # Other layouts.  The dense form sums E exponentials, in another order where a lane holds other
    # experts: the same gradients within that bound, the same bits where nothing is summed over E.
    wide_in = torch.full((T, E + 16), float("nan"), dtype=dtype, device=DEV)
    wide_in[:, 8:8 + E] = lt
    for off, ld_out in ((8, E + 24), (1, E + 5), (0, E)):
        out = torch.full((T, ld_out + off), float("nan"), dtype=dtype, device=DEV)
        view = out[:, off:off + E]
        F.moe_route_topk_backward(wide_in[:, 8:8 + E], *args, d_logits=view, **opts)
        assert out[:, :off].isnan().all() and out[:, off + E:].isnan().all()
        if scoring == "softmax" and not renormalize:
            assert (np.abs(view.double().cpu().numpy() - ref) <= bound).all()
        else:
            assert torch.equal(view, got)


# ------------------------------------------------------------------ norms: several rows a workgroup


def between_roundings(got, ref, err, what):
    """got bf16 lies between the roundings of ref - err and ref + err (rounding is monotonic)."""
    lo, hi = (ref - err).to(BF), (ref + err).to(BF)
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), "%s: %d of %d off, first at %s" % (what, bad.sum(), bad.numel(), bad.nonzero()[0].tolist())


def within(got, ref, err, what):
    bad = ~((got.double() - ref).abs() <= err)
    assert not bad.any(), "%s: %d of %d off, first at %s" % (what, bad.sum(), bad.numel(), bad.nonzero()[0].tolist())


def output(got, ref, err, what):
    (between_roundings if got.dtype == BF else within)(got, ref, err, what)


def depth(N):
    """Additions on the way of one of N terms of a row: a thread's 8 or 16, lanes (4 + 2), wavefronts (4)."""
    return (8 if N <= 8192 else 16) + 10


def inv_rel(N):
    """1 / sqrt(mean square + eps): half of the sum's, the mean's (2) and eps' (1) roundings, and two ulps of its own."""
    return ((depth(N) + 3) / 2 + 2) * U


def rows_of(seed, T, N, gate, res):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def r(*shape, dtype=BF):
        return torch.randn(shape, generator=g, device=DEV).to(dtype)
    # rows of unequal magnitudes: one taken for another does not go unnoticed
    size = torch.exp(torch.randn(T, 1, generator=g, device=DEV))
    return dict(x=(r(T, N, dtype=torch.float32) * 2 * size).to(res), y=(r(T, N, dtype=torch.float32) * size.flip(0)).to(BF),
                w_pre=1 + 0.2 * r(N), w_post=1 + 0.2 * r(N), gate=r(T, N) if gate == "full" else r(N) if gate else None,
                dz=r(T, N), dh=r(T, N, dtype=res))


MANY_ROWS = [  # T past three rows for each workgroup of the grid: with an odd remainder where T is
    (6145, 520), (3073, 2048), (769, 5120), (769, 7168), (771, 16384), (770, 8200)]
KINDS = [(BF, "channel", True), (torch.float32, "full", True), (torch.float32, "channel", False), (BF, None, True),
         (torch.float32, "before", False), (BF, "full", False)]


def parts(a, gate, post):
    kw = dict(y=None if gate == "before" else a["y"], w_post=a["w_post"] if post else None,
              gate=None if gate == "before" else a["gate"])
    return kw, (lambda rows: {n: t[rows] if t is not None and t.dim() == 2 else t for n, t in kw.items()})


@pytest.mark.parametrize("T,N", MANY_ROWS)
@pytest.mark.parametrize("res,gate,post", KINDS)
def test_norm_of_many_rows(T, N, res, gate, post):
    a = rows_of(T + N, T, N, gate, res)
    kw, part_of = parts(a, gate, post)
    out = "both" if N % 128 == 0 else "bf16"
    opts = dict(residual_scale=0.75, eps=1e-5, out=out)
    h, z, q, sf = F.residual_rms_norm(a["x"], a["w_pre"], **kw, **opts)
    again = F.residual_rms_norm(a["x"], a["w_pre"], **kw, **opts)
    assert torch.equal(h, again[0]) and torch.equal(z, again[1])
    # the same bits as calls in which no workgroup has a second row
    for t in range(0, T, 256):
        rows = slice(t, min(T, t + 256))
        n = rows.stop - t
        h1, z1, q1, sf1 = F.residual_rms_norm(a["x"][rows], a["w_pre"], **part_of(rows), **opts)
        assert torch.equal(h[rows], h1) and torch.equal(z[rows], z1), "rows from %d" % t
        if q is not None:
            assert torch.equal(q[rows], q1) and torch.equal(sf[:, rows], sf1[:, :n]), "rows from %d" % t
    # 64 bits
    x, w_pre = a["x"].double(), a["w_pre"].double()
    b = torch.zeros_like(x)
    if gate != "before":
        b = a["y"].double()
        if post:
            b = b * torch.rsqrt(b.square().mean(1, keepdim=True) + 1e-5) * a["w_post"].double()
        if a["gate"] is not None:
            b = b * a["gate"].double()
    href = 0.75 * x + b
    # b: its row's factor, the weights' two products, the products with y and a gate of the token; then one of h
    herr = (inv_rel(N) + 5 * U) * b.abs() + U * href.abs()
    output(h, href, herr, "h")
    inv = torch.rsqrt(href.square().mean(1, keepdim=True) + 1e-5)
    # h's errors move its root mean square by their own at most; the factor times the weight, and the product
    rel = herr.norm(dim=1, keepdim=True) / href.norm(dim=1, keepdim=True) + inv_rel(N) + 3 * U
    zref = href * inv * w_pre
    zerr = (herr + rel * href.abs()) * inv * w_pre.abs() * (1 + 1e-4)
    between_roundings(z, zref, zerr, "z")
    if q is not None:  # (every 37th row: the rest has the bits of short calls)
        some = torch.arange(T - 1, -1, -37, device=DEV)
        R.check_quantized(zref[some].cpu().numpy(), q[some].cpu().numpy(), sf[:, some].cpu().numpy(), zerr[some].cpu().numpy())


BACKWARD_ROWS = [(2305, 520), (705, 2048), (700, 7168), (4099, 256), (515, 16384), (513, 8200)]


@pytest.mark.parametrize("T,N", BACKWARD_ROWS)
@pytest.mark.parametrize("res,gate,post", KINDS)
def test_norm_backward_of_many_rows(T, N, res, gate, post):
    a = rows_of(T * N, T, N, gate, res)
    kw, part_of = parts(a, gate, post)
    opts = dict(residual_scale=0.75, eps=1e-5)
    got = F.residual_rms_norm_backward(a["dz"], a["x"], a["w_pre"], d_h=a["dh"], **kw, **opts)
    for g1, g2 in zip(got, F.residual_rms_norm_backward(a["dz"], a["x"], a["w_pre"], d_h=a["dh"], **kw, **opts)):
        assert g1 is None and g2 is None or torch.equal(g1, g2)
    for t in range(0, T, 256):  # (a grid has at least 256 workgroups where there are as many rows)
        rows = slice(t, min(T, t + 256))
        one = F.residual_rms_norm_backward(a["dz"][rows], a["x"][rows], a["w_pre"], d_h=a["dh"][rows], **part_of(rows), **opts)
        for name, g, g1 in zip(("d_x", "d_y", "", "", "d_gate"), got, one):
            if name and g is not None and g.dim() == 2:
                assert torch.equal(g[rows], g1), "%s, rows from %d" % (name, t)
    # 64 bits.  Sums of a row as above; a product and its weight add 2 roundings to each term of the inner products
    h, dz, dh_in, w_pre = a["x"].double(), a["dz"].double(), a["dh"].double(), a["w_pre"].double()
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    rh = torch.rsqrt(mean(h * h) + 1e-5)
    hh, u = h * rh, dz * w_pre
    m, m_abs = mean(u * hh), mean((u * hh).abs())
    m_err = (depth(N) + 6) * U * m_abs + inv_rel(N) * m.abs()
    dh = dh_in + rh * (u - hh * m)
    # u, hh * m, their difference, the factor, the sum
    dh_err = rh * ((inv_rel(N) + 4 * U) * u.abs() + hh.abs() * (m_err + (2 * inv_rel(N) + 4 * U) * m.abs())) + U * dh.abs()
    slack = 1 + 1e-4  # terms of u^2
    output(got[0], 0.75 * dh, (0.75 * dh_err + U * dh.abs()) * slack, "d_x")
    # sums over the tokens: a workgroup's rows one after the other (at most 16 here), then one in sixteen of the
    # workgroups' sums (of at most 512 here), then sixteen
    rows_depth = 16 + 512 // 16 + 16
    over_rows = lambda t, err: (t.sum(0), (err.sum(0) + rows_depth * U * t.abs().sum(0)) * slack)  # noqa: E731
    t = dz * hh
    within(got[2], *over_rows(t, (inv_rel(N) + 2 * U) * t.abs()), "d_w_pre")
    if gate == "before":
        assert got[1] is None and got[3] is None and got[4] is None
        return
    y = a["y"].double()
    gt = torch.ones_like(y) if a["gate"] is None else a["gate"].double() * torch.ones_like(y)
    db, db_err = dh * gt, dh_err * gt.abs() + U * (dh * gt).abs()
    yh, wp, ry_rel = y, torch.ones_like(w_pre), 0.0
    if post:
        wp, ry_rel = a["w_post"].double(), inv_rel(N)
        ry = torch.rsqrt(mean(y * y) + 1e-5)
        yh = y * ry
        v = db * wp
        m, m_abs = mean(v * yh), mean((v * yh).abs())
        m_err = mean((db_err * wp * yh).abs()) + (depth(N) + 8) * U * m_abs + ry_rel * m.abs()
        dy = ry * (v - yh * m)
        dy_err = ry * (db_err * wp.abs() + (ry_rel + 4 * U) * v.abs() + yh.abs() * (m_err + (2 * ry_rel + 4 * U) * m.abs()))
        output(got[1], dy, (dy_err + U * dy.abs()) * slack, "d_y")
        t = db * yh
        within(got[3], *over_rows(t, db_err * yh.abs() + (ry_rel + 2 * U) * t.abs()), "d_w_post")
    else:
        assert got[3] is None
        output(got[1], db, db_err * slack, "d_y")
    if a["gate"] is None:
        assert got[4] is None
        return
    t = dh * yh * wp
    err = dh_err * (yh * wp).abs() + (ry_rel + 3 * U) * t.abs()
    if a["gate"].dim() == 1:
        within(got[4], *over_rows(t, err), "d_gate")
    else:
        output(got[4], t, err * slack, "d_gate")


# ------------------------------------------------------------------ checkpoint: several units a wavefront

# experts, rows an expert, columns: past three (row, 512 columns) units for each of the grid's 7168 wavefronts, with
# experts that are empty, full, over-full and ragged
UNITS = [(37, 700, 640), (19, 699, 2048), (90, 501, 128)]


def many_units(E, M, H):
    g = gen(3, E, M)
    counts = g.integers(0, M + 1, E)
    counts[[0, 5, 6, E - 1]] = 0, M, M + 9, -3
    counts[7:] = np.where(g.random(E - 7) < 0.8, np.maximum(counts[7:], M - 40), counts[7:])
    valid = torch.from_numpy(np.arange(M) < np.clip(counts, 0, M)[:, None]).to(DEV)
    assert int(valid.sum()) * -(-H // 512) > 3 * 7168
    t = torch.Generator(device=DEV).manual_seed(E)
    size = torch.exp(torch.randn(E, M, 1, generator=t, device=DEV))
    x = (torch.randn(E, M, 2 * H, generator=t, device=DEV) * size).to(BF)
    x[~valid] = float("nan")
    return torch.from_numpy(counts).int().to(DEV), valid, x, t


def padding(*shape, dtype=torch.uint8):
    return torch.full(shape, 0x2B if dtype == torch.uint8 else -7, dtype=dtype, device=DEV)


def values(codes, words, groups):
    """Values of codes [E, M, 128 * groups] at the UE8M0 bytes of words [E, ceil(groups / 4), M], in 64 bits."""
    E, W, M = words.shape
    b = words.view(torch.uint8).view(E, W, M, 4).transpose(1, 2).reshape(E, M, 4 * W)[..., :groups]
    return codes.view(torch.float8_e4m3fn).double() * torch.exp2(b.double() - 127).repeat_interleave(128, dim=-1)


@pytest.mark.parametrize("E,M,H", UNITS)
def test_checkpoint_of_many_units(E, M, H):
    m, valid, x, _ = many_units(E, M, H)
    W = -(-H // 512)
    new = lambda: [padding(E, M, H), padding(E, W, M, dtype=torch.int32),  # noqa: E731
                   padding(E, M, 2 * H), padding(E, 2 * W, M, dtype=torch.int32)]
    q, sf, cq, csf = F.silu_mul_quant_group_pack_checkpoint(x, m, *new())
    for a, b in zip((q, sf, cq, csf), F.silu_mul_quant_group_pack_checkpoint(x, m, *new())):
        assert torch.equal(a, b)
    q2, sf2 = F.silu_mul_quant_group_pack(x, m, q=padding(E, M, H), sf=padding(E, W, M, dtype=torch.int32))
    assert torch.equal(q, q2) and torch.equal(sf, sf2)
    assert (cq[~valid] == 0x2B).all() and (csf.transpose(1, 2)[~valid] == -7).all()
    for half in (0, 1):  # each half value for value as a quantization of its own
        rq, rsf = F.fp8_quant_group_pack(x[..., half * H:(half + 1) * H].reshape(E * M, H).contiguous())
        assert torch.equal(cq[..., half * H:(half + 1) * H][valid], rq.view(E, M, H)[valid])
        rows = csf[:, half * W:(half + 1) * W].transpose(1, 2)[valid]
        assert torch.equal(rows, rsf[:, :E * M].t().reshape(E, M, W)[valid])


@pytest.mark.parametrize("E,M,H", UNITS)
def test_checkpoint_backward_of_many_units(E, M, H):
    m, valid, x, t = many_units(E, M, H)
    W, W2 = -(-H // 512), -(-2 * H // 512)
    _, _, cq, csf = F.silu_mul_quant_group_pack_checkpoint(x, m)
    d = torch.randn(E, M, H, generator=t, device=DEV).to(BF)
    d[~valid] = float("nan")
    dx = F.silu_mul_backward_from_checkpoint(d, m, cq, csf, d_x=torch.full_like(x, float("nan")))
    q, sf = F.silu_mul_backward_from_checkpoint(d, m, cq, csf, quantize=True, q=padding(E, M, 2 * H),
                                                sf=padding(E, W2, M, dtype=torch.int32))
    assert dx[~valid].isnan().all() and (q[~valid] == 0x2B).all() and (sf.transpose(1, 2)[~valid] == -7).all()
    # the same bits as an expert alone, where no wavefront has a second unit
    for e in range(E):
        one = slice(e, e + 1)
        n = int(valid[e].sum())
        assert n * W <= 7168
        dx1 = F.silu_mul_backward_from_checkpoint(d[one], m[one], cq[one], csf[one])
        assert torch.equal(dx[e, :n], dx1[0, :n]), "expert %d" % e
        q1, sf1 = F.silu_mul_backward_from_checkpoint(d[one], m[one], cq[one], csf[one], quantize=True)
        assert torch.equal(q[e, :n], q1[0, :n]) and torch.equal(sf[e, :, :n], sf1[0, :, :n]), "expert %d" % e
    # 64 bits
    groups = H // 128
    cs = csf.view(E, 2, W, M)
    gate = values(cq[..., :H].contiguous(), cs[:, 0].contiguous(), groups)[valid]
    up = values(cq[..., H:].contiguous(), cs[:, 1].contiguous(), groups)[valid]
    s, rest, dv = torch.sigmoid(gate), torch.sigmoid(-gate), d[valid].double()
    ref = torch.cat([dv * up * s * (1 + gate * rest), dv * gate * s], -1)
    # exp of a rounded argument, reciprocal, four products: 16 roundings, of 1 + |gate| (1 - s) where gates are negative
    err = 16 * U * torch.cat([(dv * up).abs() * s * (1 + gate.abs() * rest), (dv * gate).abs() * s], -1) + 1e-36
    between_roundings(dx[valid], ref, err, "d_x")
    some = torch.arange(ref.shape[0] - 1, -1, -37, device=DEV)
    rows = sf.transpose(1, 2)[valid][some].t().contiguous()
    R.check_quantized(ref[some].cpu().numpy(), q[valid][some].cpu().numpy(), rows.cpu().numpy(), err[some].cpu().numpy())
