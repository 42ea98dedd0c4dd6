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
