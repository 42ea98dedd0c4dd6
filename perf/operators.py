"""Cases of the operators around the FP8 experts' products: routing, combine, the norms of
the residual stream, and the 8-bit checkpoint of the gated activation, each with its
backward pass.

`run` computes them in plain torch operations, or, where `own` is true, with the calls a
user of block_scaled_fp8_token_amd makes.  Codes of 8 bits and their scales are returned
as tensors of the 8-bit float types that they are (e4m3, and e8m0 for the UE8M0 bytes).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step: sigmoid scores, balance bias, 4 of 8 groups of experts
        dict(name="route_token", op="route", tokens=1, experts=256, topk=8, groups=8, topk_groups=4, group_top=2,
             scoring="sigmoid", bias=True, renormalize=True, logits="float32"),
        # a prompt batch through the same router, logits as a bf16 product left them
        dict(name="route_prompt", op="route", tokens=16384, experts=256, topk=8, groups=8, topk_groups=4, group_top=2,
             scoring="sigmoid", bias=True, renormalize=True, logits="bfloat16"),
        # training step of a softmax router without renormalisation: every logit has a gradient
        dict(name="route_backward", op="route_backward", tokens=8193, experts=160, topk=6, scoring="softmax",
             renormalize=False, logits="float32"),
        # decode batch: 64 tokens, eight rows each, on top of the shared path's output
        dict(name="combine_decode", op="combine", tokens=64, topk=8, experts=32, cols=7168, base=True),
        # prompt batch
        dict(name="combine_prompt", op="combine", tokens=4096, topk=8, experts=32, cols=7168, base=True),
        # training step: rows' gradients quantised for the experts' next product, weights' gradients
        dict(name="combine_backward", op="combine_backward", tokens=2048, topk=8, experts=32, cols=7168, quantize=True),
        # one decode token between two blocks: bf16 for the router, e4m3 for the experts
        dict(name="norm_token", op="norm", tokens=1, cols=7168, post=True, gate="channel", residual="bfloat16",
             out="both"),
        # prompt batch feeding an FP8 product
        dict(name="norm_prompt", op="norm", tokens=8192, cols=7168, post=True, gate="channel", residual="bfloat16",
             out="fp8"),
        # training step over an odd number of tokens, residual stream in fp32
        dict(name="norm_backward", op="norm_backward", tokens=4097, cols=7168, post=True, gate="channel",
             residual="float32"),
        # small training microbatch through 32 experts padded to 256 rows
        dict(name="silu_small", op="silu", rows=512, experts=32, capacity=256, half=2048),
        # large training microbatch
        dict(name="silu_large", op="silu", rows=32768, experts=32, capacity=2048, half=2048),
        # its backward pass from the 8-bit checkpoint
        dict(name="silu_backward", op="silu_backward", rows=32768, experts=32, capacity=2048, half=2048,
             quantize=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "combine", "combine_backward", "norm", "norm_backward", "silu",
                     "silu_backward"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.randint(max(2, 32 // groups), 256 // groups)
        scoring = rng.choice(["sigmoid", "softmax"])
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, topk=rng.randint(1, 8), groups=groups,
                    topk_groups=max(1, groups // 2), group_top=2 if scoring == "sigmoid" and groups > 1 else 1,
                    scoring=scoring, bias=scoring == "sigmoid" and rng.random() < 0.7,
                    renormalize=rng.random() < 0.7, logits=rng.choice(["float32", "bfloat16"]))
    if op == "route_backward":
        return dict(op=op, tokens=_log(rng, 1, 8192), experts=rng.randint(16, 256), topk=rng.randint(2, 8),
                    scoring=rng.choice(["sigmoid", "softmax"]), renormalize=rng.random() < 0.6,
                    logits=rng.choice(["float32", "bfloat16"]))
    if op == "combine":
        return dict(op=op, tokens=_log(rng, 1, 4096), topk=rng.randint(1, 8), experts=rng.randint(8, 64),
                    cols=8 * rng.randint(64, 896), base=rng.random() < 0.5)
    if op == "combine_backward":
        quantize = rng.random() < 0.5
        return dict(op=op, tokens=_log(rng, 1, 2048), topk=rng.randint(1, 8), experts=rng.randint(8, 64),
                    cols=128 * rng.randint(4, 56) if quantize else 8 * rng.randint(64, 896), quantize=quantize)
    if op == "norm":
        out = rng.choice(["bf16", "fp8", "both"])
        return dict(op=op, tokens=_log(rng, 1, 8192), cols=8 * rng.randint(64, 896) if out == "bf16" else 128 * rng.randint(4, 56),
                    post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "full"]),
                    residual=rng.choice(["bfloat16", "float32"]) if out == "fp8" else "bfloat16", out=out)
    if op == "norm_backward":
        return dict(op=op, tokens=_log(rng, 1, 4097), cols=8 * rng.randint(64, 800), post=rng.random() < 0.7,
                    gate=rng.choice(["none", "channel", "full"]), residual=rng.choice(["bfloat16", "float32"]))
    experts = rng.randint(1, 64)
    rows = _log(rng, 1, 24576)
    case = dict(op=op, rows=rows, experts=experts, capacity=max(8, -(-rows * 2 // experts)), half=128 * rng.randint(2, 16))
    if op == "silu_backward":
        case["quantize"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _routing(g, T, k, E):
    """ids [T, k] distinct in a row, of experts of unequal popularity (one pair in 64 names none), slots in pair order."""
    pop = torch.randn(E, generator=g, device=DEV) * 0.2
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp(1e-7, 1 - 1e-6)))
    ids = (pop + noise).topk(k, dim=1).indices.reshape(-1)
    ids[37::64] = E
    order = torch.sort(ids, stable=True).indices
    ids_sorted = ids[order]
    starts = torch.cumsum(torch.bincount(ids, minlength=E + 1), 0) - torch.bincount(ids, minlength=E + 1)
    slots = torch.empty_like(ids)
    slots[order] = torch.arange(T * k, device=DEV) - starts[ids_sorted]
    capacity = _capacity(T, k, E)
    none = (ids == E) | (slots >= capacity)
    ids = torch.where(ids == E, -1, ids)
    slots = torch.where(none, -1, slots)
    return ids.view(T, k).int(), slots.view(T, k).int()


def _capacity(T, k, E):
    return min(T, -(-2 * T * k // E) + 8)


def _counts(seed, rows, E, capacity):
    """Rows per expert, Zipf-skewed, none past the capacity, `rows` in all."""
    rng = np.random.default_rng([seed, 11])
    p = np.arange(1, E + 1) ** -0.5
    counts = np.minimum(rng.multinomial(rows, p / p.sum()), capacity)
    left = rows - counts.sum()
    for e in rng.permutation(E):
        more = min(left, capacity - counts[e])
        counts[e] += more
        left -= more
    return torch.from_numpy(counts.astype(np.int32)).to(DEV)


def _quant(v):
    """1x128 groups along the last dimension: (e4m3 codes, UE8M0 bytes [..., groups]); the exponent is the smallest
    with 448 * 2^e >= the group's largest magnitude, at least -42."""
    grouped = v.unflatten(-1, (-1, 128))
    m, x = torch.frexp(grouped.abs().amax(-1))
    e = torch.where(m > 0, x - 9 + (m > 0.875), -42).clamp(min=-42)
    codes = (grouped * torch.exp2(-e.float()).unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2)
    return codes, (e + 127).to(torch.uint8)


def _words(b):
    """UE8M0 bytes [..., rows, groups] as the packed words' bytes [..., words, 4 * rows] (four groups of a row to a word)."""
    pad = -b.shape[-1] % 4
    if pad:
        b = torch.cat([b, torch.zeros(*b.shape[:-1], pad, dtype=b.dtype, device=b.device)], -1)
    return b.unflatten(-1, (-1, 4)).transpose(-2, -3).flatten(-2)


def _checkpoint(x):
    """gate and up halves of x [E, M, 2H] in 8 bits: codes [E, M, 2H], words' bytes [E, 2 * words(H), 4 * M]."""
    H = x.shape[-1] // 2
    gc, gs = _quant(x[..., :H])
    uc, us = _quant(x[..., H:])
    return torch.cat([gc.view(torch.uint8), uc.view(torch.uint8)], -1), torch.cat([_words(gs), _words(us)], -2)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, k = case["tokens"], case["experts"], case["topk"]
        s["l"] = _normal(g, (T, E), 1.5, getattr(torch, case["logits"]))
        if op == "route":
            # the bias moves in steps of 1e-3, as balance updates leave it
            s["b"] = torch.randint(-50, 51, (E,), generator=g, device=DEV).float() * 1e-3 if case["bias"] else None
        else:
            s["ids"] = torch.topk(s["l"].float(), k, dim=1).indices.int()
            s["dw"] = _normal(g, (T, k), 1.0, torch.float32)
    elif op in ("combine", "combine_backward"):
        T, k, E, N = case["tokens"], case["topk"], case["experts"], case["cols"]
        M = s["capacity"] = _capacity(T, k, E)
        s["ids"], s["slots"] = _routing(g, T, k, E)
        w = torch.rand(T, k, generator=g, device=DEV) + 0.1
        s["w"] = w / w.sum(1, keepdim=True)
        s["y"] = _normal(g, (E, M, N))
        if op == "combine":
            s["base"] = _normal(g, (T, N)) if case["base"] else None
        else:
            s["dout"] = _normal(g, (T, N), 1e-2)
            # one row more than the layout has: where the plain form puts the pairs that have no slot
            if case["quantize"]:
                s["q"] = torch.zeros(E * M + 1, N, dtype=torch.uint8, device=DEV)
                s["sf"] = torch.zeros(E, -(-N // 512), M, dtype=torch.int32, device=DEV)
            else:
                s["dy"] = torch.zeros(E * M + 1, N, dtype=torch.bfloat16, device=DEV)
    elif op in ("norm", "norm_backward"):
        T, N = case["tokens"], case["cols"]
        res = getattr(torch, case["residual"])
        s["y"] = _normal(g, (T, N), 0.5)
        s["w_post"] = _normal(g, (N,), 0.1) + 1 if case["post"] else None
        s["w_pre"] = _normal(g, (N,), 0.1) + 1
        s["gate"] = {"none": None, "channel": lambda: _normal(g, (N,), 0.3), "full": lambda: _normal(g, (T, N), 0.3)}[case["gate"]]
        s["gate"] = s["gate"]() if s["gate"] else None
        s["scale"] = 0.9
        if op == "norm":
            s["x"] = _normal(g, (T, N), 2.0, res)
        else:
            s["h"] = _normal(g, (T, N), 2.0, res)
            s["dh"] = _normal(g, (T, N), 1e-2, res)
            s["dz"] = _normal(g, (T, N), 1e-2)
    else:
        E, M, H = case["experts"], case["capacity"], case["half"]
        s["m"] = _counts(seed, case["rows"], E, M)
        x = _normal(g, (E, M, 2 * H))
        word_rows = -(-H // 512)
        if op == "silu":
            s["x"] = x
            s["q"] = torch.zeros(E, M, H, dtype=torch.uint8, device=DEV)
            s["sf"] = torch.zeros(E, word_rows, M, dtype=torch.int32, device=DEV)
            s["cq"] = torch.zeros(E, M, 2 * H, dtype=torch.uint8, device=DEV)
            s["csf"] = torch.zeros(E, 2 * word_rows, M, dtype=torch.int32, device=DEV)
        else:
            cq, cs = _checkpoint(x)
            s["cq"], s["csf"] = cq, cs.contiguous().view(torch.int32)
            s["dy"] = _normal(g, (E, M, H), 1e-2)
            if case["quantize"]:
                s["q"] = torch.zeros(E, M, 2 * H, dtype=torch.uint8, device=DEV)
                s["sf"] = torch.zeros(E, -(-2 * H // 512), M, dtype=torch.int32, device=DEV)
            else:
                s["dx"] = torch.zeros(E, M, 2 * H, dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------- one pass

SCALE = 2.5  # of the routing weights


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _e4m3(q):
    return q.view(torch.float8_e4m3fn)


def _e8m0(sf, rows):
    return sf[..., :rows].view(torch.float8_e8m0fnu)


def _plain_route(s):
    l = s["l"].float()
    T, E = l.shape
    k, G = s["topk"], s["groups"]
    if s["scoring"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
        key = l if s["b"] is None else score + s["b"]
        two = score if s["b"] is None else key
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
        key = two = l
    if G > 1:
        if s["group_top"] == 1:
            group = key.view(T, G, -1).amax(-1)
        else:
            best = torch.sort(two.view(T, G, -1), dim=-1, descending=True).values
            group = best[..., 0] + best[..., 1]
        kept = torch.sort(group, dim=-1, descending=True, stable=True).indices[:, : s["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter(1, kept, True)
        key = torch.where(keep.repeat_interleave(E // G, dim=1), key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    ids = order.indices[:, :k]
    some = order.values[:, :k] > -math.inf
    w = torch.where(some, score.gather(1, ids), 0)
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return torch.where(some, ids, -1).int(), w * SCALE


def _own_route(s):
    import block_scaled_fp8_token_amd as F
    return F.moe_route_topk(s["l"], s["topk"], bias=s["b"], groups=s["groups"], topk_groups=s["topk_groups"],
                            group_top=s["group_top"], scoring=s["scoring"], renormalize=s["renormalize"], scale=SCALE)


def _plain_route_backward(s):
    l, ids, dw = s["l"].float(), s["ids"].long(), s["dw"]
    if s["scoring"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    sel = score.gather(1, ids)
    if s["renormalize"]:
        r = sel / sel.sum(1, keepdim=True)
        ds = SCALE * (dw - (dw * r).sum(1, keepdim=True)) / sel.sum(1, keepdim=True)
    else:
        ds = SCALE * dw
    ds = torch.zeros_like(l).scatter(1, ids, ds)
    if s["scoring"] == "sigmoid":
        dl = ds * score * (1 - score)
    elif s["renormalize"]:  # a softmax over the selected logits: its inner sum is zero
        dl = ds * score
    else:
        dl = score * (ds - (ds * score).sum(1, keepdim=True))
    return dl.to(s["l"].dtype)


def _own_route_backward(s):
    import block_scaled_fp8_token_amd as F
    return F.moe_route_topk_backward(s["l"], s["ids"], s["dw"], scoring=s["scoring"], renormalize=s["renormalize"],
                                     scale=SCALE)


def _place(s):
    """Row of every pair in the experts' layout, and whether it has one."""
    ids, slots = s["ids"].long(), s["slots"].long()
    return ids * s["capacity"] + slots, slots >= 0


def _plain_combine(s):
    row, some = _place(s)
    rows = s["y"].flatten(0, 1)[row.clamp(min=0)].float()
    out = (rows * torch.where(some, s["w"], 0).unsqueeze(-1)).sum(1)
    if s["base"] is not None:
        out = out + s["base"].float()
    return out.to(torch.bfloat16)


def _own_combine(s):
    import block_scaled_fp8_token_amd as F
    return F.moe_combine(s["y"], s["ids"], s["slots"], weights=s["w"], base=s["base"])


def _plain_combine_backward(s):
    row, some = _place(s)
    E, M = s["experts"], s["capacity"]
    dout = s["dout"].float().unsqueeze(1)
    dw = torch.where(some, (s["y"].flatten(0, 1)[row.clamp(min=0)].float() * dout).sum(-1), 0)
    dy = dout * s["w"].unsqueeze(-1)
    to = torch.where(some, row, E * M)
    if not s["quantize"]:
        s["dy"][to] = dy.to(torch.bfloat16)
        return s["dy"][:-1].view(E, M, -1), dw
    codes, b = _quant(dy)
    s["q"][to] = codes.view(torch.uint8)
    groups = torch.zeros(E * M + 1, b.shape[-1], dtype=torch.uint8, device=b.device)
    groups[to] = b
    sf = _words(groups[:-1].view(E, M, -1)).contiguous().view(torch.int32)
    return _e4m3(s["q"][:-1].view(E, M, -1)), _e8m0(sf, M), dw


def _own_combine_backward(s):
    import block_scaled_fp8_token_amd as F
    E, M = s["experts"], s["capacity"]
    if not s["quantize"]:
        return F.moe_combine_backward(s["dout"], s["y"], s["ids"], s["slots"], weights=s["w"],
                                      d_y=s["dy"][:-1].view(E, M, -1))
    q, sf, dw = F.moe_combine_backward(s["dout"], s["y"], s["ids"], s["slots"], weights=s["w"], quantize=True,
                                       q=s["q"][:-1].view(E, M, -1), sf=s["sf"])
    return _e4m3(q), _e8m0(sf, M), dw


def _unit(v):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    branch = s["y"].float()
    if s["w_post"] is not None:
        branch = _unit(branch) * s["w_post"].float()
    if s["gate"] is not None:
        branch = branch * s["gate"].float()
    h = s["scale"] * s["x"].float() + branch
    z = _unit(h) * s["w_pre"].float()
    got = [h.to(s["x"].dtype)]
    if s["out"] != "fp8":
        got.append(z.to(torch.bfloat16))
    if s["out"] != "bf16":
        codes, b = _quant(z)
        got += [codes, _words(b).contiguous().view(torch.float8_e8m0fnu)]
    return got


def _own_norm(s):
    import block_scaled_fp8_token_amd as F
    h, z, q, sf = F.residual_rms_norm(s["x"], s["w_pre"], y=s["y"], w_post=s["w_post"], gate=s["gate"],
                                      residual_scale=s["scale"], eps=EPS, out=s["out"])
    got = [h]
    if z is not None:
        got.append(z)
    if q is not None:
        got += [_e4m3(q), _e8m0(sf, s["tokens"])]
    return got


def _plain_norm_backward(s):
    h, y, dz = s["h"].float(), s["y"].float(), s["dz"].float()
    rh = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    hh = h * rh
    u = dz * s["w_pre"].float()
    dh = s["dh"].float() + rh * (u - hh * (u * hh).mean(-1, keepdim=True))
    got = {"x": (s["scale"] * dh).to(s["h"].dtype), "w_pre": (dz * hh).sum(0)}
    branch = y
    if s["w_post"] is not None:
        ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        yh = y * ry
        branch = yh * s["w_post"].float()
    db = dh
    if s["gate"] is not None:
        db = dh * s["gate"].float()
        got["gate"] = (dh * branch).sum(0) if s["gate"].dim() == 1 else (dh * branch).to(torch.bfloat16)
    if s["w_post"] is not None:
        got["w_post"] = (db * yh).sum(0)
        v = db * s["w_post"].float()
        db = ry * (v - yh * (v * yh).mean(-1, keepdim=True))
    got["y"] = db.to(torch.bfloat16)
    return got


def _own_norm_backward(s):
    import block_scaled_fp8_token_amd as F
    dx, dy, dw_pre, dw_post, dgate = F.residual_rms_norm_backward(
        s["dz"], s["h"], s["w_pre"], d_h=s["dh"], y=s["y"], w_post=s["w_post"], gate=s["gate"],
        residual_scale=s["scale"], eps=EPS)
    got = {"x": dx, "y": dy, "w_pre": dw_pre, "w_post": dw_post, "gate": dgate}
    return {n: t for n, t in got.items() if t is not None}


def _valid(s):
    """[E, M, 1]: whether a row is one of its expert's."""
    return (torch.arange(s["capacity"], device=s["m"].device) < s["m"].unsqueeze(1)).unsqueeze(-1)


def _plain_silu(s):
    x, H = s["x"].float(), s["half"]
    gate, up = x[..., :H], x[..., H:]
    codes, b = _quant(gate / (1 + torch.exp(-gate)) * up)
    cq, cs = _checkpoint(x)
    ok = _valid(s)
    some = ok.squeeze(-1).unsqueeze(1).repeat_interleave(4, dim=-1)
    z8 = torch.zeros((), dtype=torch.uint8, device=x.device)
    q = torch.where(ok, codes.view(torch.uint8), z8)
    cq = torch.where(ok, cq, z8)
    return (_e4m3(q), torch.where(some, _words(b), z8).view(torch.float8_e8m0fnu), _e4m3(cq),
            torch.where(some, cs, z8).view(torch.float8_e8m0fnu))


def _own_silu(s):
    import block_scaled_fp8_token_amd as F
    q, sf, cq, csf = F.silu_mul_quant_group_pack_checkpoint(s["x"], s["m"], q=s["q"], sf=s["sf"], cq=s["cq"],
                                                            csf=s["csf"])
    M = s["capacity"]
    return _e4m3(q), _e8m0(sf, M), _e4m3(cq), _e8m0(csf, M)


def _decode_checkpoint(s, dtype):
    """gate and up [E, M, H] from the codes and the words' bytes."""
    H, E, M = s["half"], s["experts"], s["capacity"]
    b = s["csf"].view(torch.uint8).view(E, 2, -1, M, 4).transpose(2, 3).flatten(3)[..., : H // 128]
    values = torch.exp2(b.to(dtype) - 127).repeat_interleave(128, dim=-1)  # [E, 2, M, H]
    codes = _e4m3(s["cq"]).to(dtype)
    return codes[..., :H] * values[:, 0], codes[..., H:] * values[:, 1]


def _plain_silu_backward(s):
    gate, up = _decode_checkpoint(s, torch.float32)
    dy = s["dy"].float()
    sg = 1 / (1 + torch.exp(-gate))
    dx = torch.cat([dy * up * sg * (1 + gate * (1 - sg)), dy * gate * sg], -1)
    ok = _valid(s)
    if not s["quantize"]:
        return torch.where(ok, dx, 0).to(torch.bfloat16)
    codes, b = _quant(dx)
    some = ok.squeeze(-1).unsqueeze(1).repeat_interleave(4, dim=-1)
    z8 = torch.zeros((), dtype=torch.uint8, device=dx.device)
    return (_e4m3(torch.where(ok, codes.view(torch.uint8), z8)),
            torch.where(some, _words(b), z8).view(torch.float8_e8m0fnu))


def _own_silu_backward(s):
    import block_scaled_fp8_token_amd as F
    if not s["quantize"]:
        return F.silu_mul_backward_from_checkpoint(s["dy"], s["m"], s["cq"], s["csf"], d_x=s["dx"])
    q, sf = F.silu_mul_backward_from_checkpoint(s["dy"], s["m"], s["cq"], s["csf"], quantize=True, q=s["q"], sf=s["sf"])
    return _e4m3(q), _e8m0(sf, s["capacity"])


_plain = dict(route=_plain_route, route_backward=_plain_route_backward, combine=_plain_combine,
              combine_backward=_plain_combine_backward, norm=_plain_norm, norm_backward=_plain_norm_backward,
              silu=_plain_silu, silu_backward=_plain_silu_backward)
_own = dict(route=_own_route, route_backward=_own_route_backward, combine=_own_combine,
            combine_backward=_own_combine_backward, norm=_own_norm, norm_backward=_own_norm_backward, silu=_own_silu,
            silu_backward=_own_silu_backward)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, k = case["tokens"], case["experts"], case["topk"]
        n = 4 if case["logits"] == "float32" else 2
        if op == "route":  # logits, bias, ids and weights; score and bias of each expert, one comparison per expert and choice
            return {"bytes": T * E * n + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": T * E * (5 + k)}
        return {"bytes": 2 * T * E * n + 8 * T * k, "flops": T * E * 8}
    if op in ("combine", "combine_backward"):
        T, k, N = case["tokens"], case["topk"], case["cols"]
        pairs = T * k - len(range(37, T * k, 64))
        if op == "combine":
            return {"bytes": 2 * N * (pairs + T + (T if case["base"] else 0)) + 12 * T * k, "flops": 2 * pairs * N}
        out = pairs * N * (1 + 1 / 128 if case["quantize"] else 2)
        return {"bytes": 2 * N * (pairs + T) + out + 16 * T * k, "flops": (6 if case["quantize"] else 3) * pairs * N}
    if op in ("norm", "norm_backward"):
        T, N = case["tokens"], case["cols"]
        r = 4 if case["residual"] == "float32" else 2
        gate = {"none": 0, "channel": 2 * N, "full": 2 * T * N}[case["gate"]]
        weights = 2 * N * (2 if case["post"] else 1)
        if op == "norm":
            z = {"bf16": 2, "fp8": 1 + 1 / 128, "both": 3 + 1 / 128}[case["out"]]
            return {"bytes": T * N * (2 * r + 2 + z) + gate + weights, "flops": 12 * T * N}
        return {"bytes": T * N * (3 * r + 6) + (2 * gate if case["gate"] == "full" else 3 * gate) + 3 * weights, "flops": 24 * T * N}
    rows, H = case["rows"], case["half"]
    codes = 2 * H * (1 + 1 / 128)
    if op == "silu":
        return {"bytes": rows * (4 * H + 1.5 * codes), "flops": 16 * rows * H}
    return {"bytes": rows * (2 * H + codes + (codes if case["quantize"] else 4 * H)), "flops": 16 * rows * H}


# ---------------------------------------------------------------- the definitions in 64 bits

def _e4m3_grid(v):
    """The e4m3 value nearest to v (|v| <= 448), ties to the even code."""
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3)
    return torch.round(v / step) * step


def _codes_and_scales(v):
    """e4m3 values and power-of-two scales of 1x128 groups, the scales laid out as the words' bytes."""
    g = v.reshape(*v.shape[:-1], -1, 128)
    need = g.abs().amax(-1).clamp(min=1e-10) / 448
    e = torch.ceil(torch.log2(need))
    e = torch.where(torch.exp2(e - 1) >= need, e - 1, e)
    codes = _e4m3_grid(g / torch.exp2(e).unsqueeze(-1)).reshape(v.shape)
    groups = e.shape[-1]
    padded = torch.full((*e.shape[:-1], -(-groups // 4) * 4), 2.0 ** -127, dtype=v.dtype, device=v.device)
    padded[..., :groups] = torch.exp2(e)
    rows = e.shape[-2]
    return codes, padded.reshape(*e.shape[:-1], -1, 4).movedim(-2, -3).reshape(*e.shape[:-2], -1, 4 * rows)


def _exact_route(s):
    l = s["l"].double()
    T, E = l.shape
    score = torch.sigmoid(l) if s["scoring"] == "sigmoid" else torch.softmax(l, 1)
    rank = score + (s["b"].double() if s["b"] is not None else 0)
    if s["groups"] > 1:
        size = E // s["groups"]
        group = rank.reshape(T, s["groups"], size).topk(s["group_top"], dim=2).values.sum(2)
        # a group's place among the groups: those with a better score, or the same score and a lower index
        index = torch.arange(s["groups"], device=DEV)
        ahead = (group.unsqueeze(1) > group.unsqueeze(2)) | (
            (group.unsqueeze(1) == group.unsqueeze(2)) & (index.view(1, 1, -1) < index.view(1, -1, 1)))
        out = ahead.sum(2) >= s["topk_groups"]
        rank = rank.masked_fill(out.unsqueeze(2).expand(-1, -1, size).reshape(T, E), -math.inf)
    ids = rank.topk(s["topk"], dim=1).indices
    w = score.gather(1, ids)
    return None, SCALE * (w / w.sum(1, keepdim=True) if s["renormalize"] else w)


def _exact_route_backward(s):
    l = s["l"].double().requires_grad_(True)
    score = torch.sigmoid(l) if s["scoring"] == "sigmoid" else torch.softmax(l, 1)
    w = score.gather(1, s["ids"].long())
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return torch.autograd.grad((SCALE * w * s["dw"].double()).sum(), l)[0]


def _exact_combine(s):
    T, k = s["ids"].shape
    out = torch.zeros(T, s["cols"], dtype=torch.float64, device=DEV) if s["base"] is None else s["base"].double()
    for j in range(k):
        e, r = s["ids"][:, j].long(), s["slots"][:, j].long()
        has = ((r >= 0) & (e >= 0)).unsqueeze(1)
        out = out + torch.where(has, s["w"][:, j : j + 1].double() * s["y"][e.clamp(min=0), r.clamp(min=0)].double(), 0.0)
    return out


def _exact_combine_backward(s):
    E, M, N = s["experts"], s["capacity"], s["cols"]
    t, j = torch.nonzero(s["slots"] >= 0, as_tuple=True)
    e, r = s["ids"][t, j].long(), s["slots"][t, j].long()
    dw = torch.zeros(s["ids"].shape, dtype=torch.float64, device=DEV)
    dout = s["dout"].double()
    dw[t, j] = (s["y"][e, r].double() * dout[t]).sum(1)
    rows = s["w"][t, j].double().unsqueeze(1) * dout[t]
    if not s["quantize"]:
        dy = torch.zeros(E, M, N, dtype=torch.float64, device=DEV)
        dy[e, r] = rows
        return dy, dw
    codes, scales = _codes_and_scales(rows)
    q = torch.zeros(E, M, N, dtype=torch.float32, device=DEV)
    q[e, r] = codes.float()
    sf = torch.full((E, M, scales.shape[0], 4), 2.0 ** -127, dtype=torch.float64, device=DEV)
    sf[e, r] = scales.reshape(scales.shape[0], -1, 4).transpose(0, 1)
    return q, sf.movedim(2, 1).reshape(E, -1, 4 * M), dw


def _exact_norm(s):
    def normed(v, w):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * w.double()

    p = s["y"].double()
    p = p if s["w_post"] is None else normed(p, s["w_post"])
    p = p if s["gate"] is None else p * s["gate"].double()
    h = s["x"].double() * s["scale"] + p
    z = normed(h, s["w_pre"])
    got = [h]
    if s["out"] in ("bf16", "both"):
        got.append(z)
    if s["out"] in ("fp8", "both"):
        got.extend(_codes_and_scales(z))
    return got


def _exact_norm_backward(s):
    def normed(v, w):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * w

    leaf = {n: s[n].double().requires_grad_(True) for n in ("y", "w_post", "gate", "w_pre") if s[n] is not None}
    h = s["h"].double().requires_grad_(True)
    dh = s["dh"].double() + torch.autograd.grad(
        (normed(h, leaf["w_pre"]) * s["dz"].double()).sum(), [h, leaf["w_pre"]], retain_graph=True)[0]
    got = {"x": s["scale"] * dh,
           "w_pre": torch.autograd.grad((normed(h.detach(), leaf["w_pre"]) * s["dz"].double()).sum(), leaf["w_pre"])[0]}
    branch = leaf["y"] if "w_post" not in leaf else normed(leaf["y"], leaf["w_post"])
    branch = branch if "gate" not in leaf else branch * leaf["gate"]
    names = [n for n in ("y", "w_post", "gate") if n in leaf]
    got.update(zip(names, torch.autograd.grad((branch * dh).sum(), [leaf[n] for n in names])))
    return got


def _exact_silu(s):
    H, E, M = s["half"], s["experts"], s["capacity"]
    parts = [torch.zeros(E, M, H, dtype=torch.float32, device=DEV), None,
             torch.zeros(E, M, 2 * H, dtype=torch.float32, device=DEV), None]
    words = -(-H // 512)
    parts[1] = torch.full((E, words, 4 * M), 2.0 ** -127, dtype=torch.float64, device=DEV)
    parts[3] = torch.full((E, 2 * words, 4 * M), 2.0 ** -127, dtype=torch.float64, device=DEV)
    for e, n in enumerate(s["m"].tolist()):
        if n:
            gate, up = s["x"][e, :n, :H].double(), s["x"][e, :n, H:].double()
            c, b = _codes_and_scales(gate * torch.sigmoid(gate) * up)
            parts[0][e, :n], parts[1][e, :, : 4 * n] = c.float(), b
            (gc, gb), (uc, ub) = _codes_and_scales(gate), _codes_and_scales(up)
            parts[2][e, :n] = torch.cat([gc, uc], 1).float()
            parts[3][e, :words, : 4 * n], parts[3][e, words:, : 4 * n] = gb, ub
    return tuple(parts)


def _exact_silu_backward(s):
    H, E, M = s["half"], s["experts"], s["capacity"]
    gate, up = _decode_checkpoint(s, torch.float64)
    dx = torch.zeros(E, M, 2 * H, dtype=torch.float64, device=DEV)
    for e, n in enumerate(s["m"].tolist()):
        g, dy = gate[e, :n], s["dy"][e, :n].double()
        sg = torch.sigmoid(g)
        dx[e, :n, :H] = dy * up[e, :n] * (sg + g * sg * torch.sigmoid(-g))
        dx[e, :n, H:] = dy * g * sg
    if not s["quantize"]:
        return dx
    q = torch.zeros(E, M, 2 * H, dtype=torch.float32, device=DEV)
    sf = torch.full((E, -(-2 * H // 512), 4 * M), 2.0 ** -127, dtype=torch.float64, device=DEV)
    for e, n in enumerate(s["m"].tolist()):
        if n:
            c, b = _codes_and_scales(dx[e, :n])
            q[e, :n], sf[e, :, : 4 * n] = c.float(), b
    return q, sf


_exact = dict(route=_exact_route, route_backward=_exact_route_backward, combine=_exact_combine,
              combine_backward=_exact_combine_backward, norm=_exact_norm, norm_backward=_exact_norm_backward,
              silu=_exact_silu, silu_backward=_exact_silu_backward)


def exact(case, seed):
    return _exact[case["op"]](prepare(case, seed))
