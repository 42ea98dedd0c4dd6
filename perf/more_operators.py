"""Cases of the operators of a decode step: a whole mixture-of-experts layer for a few tokens
(on the e4m3 weights of the masked products, plain or pre-shuffled, and on 4-bit ones), and
products of a few rows with weights of 4 bits under group scales.

`run` computes them in plain torch operations, or, where `own` is true, with the calls a
user of block_scaled_fp8_token_amd makes.  `prepare` makes the weights in row order and in
the library's pre-shuffled order, as a program that serves a model lays them out once.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a test-sized layer, one token: what a call costs when there is next to nothing to read
        dict(name="moe_small", op="moe", tokens=1, experts=8, ranks=1, topk=2, hidden=512, half=256, weights="plain",
             base=True),
        # one token of a decode step through eight of the 32 experts that a GPU holds
        dict(name="moe_token", op="moe", tokens=1, experts=32, ranks=1, topk=8, hidden=7168, half=2048,
             weights="preshuffled", base=True),
        # 16 sequences of a decode step, half of whose choices are experts of another GPU
        dict(name="moe_share", op="moe", tokens=16, experts=32, ranks=2, topk=8, hidden=7168, half=2048,
             weights="plain", base=False),
        # 64 sequences: every expert is read, by about 16 rows
        dict(name="moe_batch", op="moe", tokens=64, experts=32, ranks=1, topk=8, hidden=7168, half=2048,
             weights="preshuffled", base=True),
        # one token, experts in 4 bits (e2m1 under power-of-two scales of 32)
        dict(name="moe_w4_token", op="moe", tokens=1, experts=32, ranks=1, topk=8, hidden=7168, half=2048,
             weights="w4", base=True),
        # an odd batch through 4-bit experts
        dict(name="moe_w4_batch", op="moe", tokens=33, experts=32, ranks=1, topk=8, hidden=7168, half=2048,
             weights="w4", base=False),
        # the smallest product of the repository's decode shapes
        dict(name="gemv_small", op="gemv", tokens=1, rows=512, cols=512, format="e2m1", group=32, zeros=False),
        # one token through the dense decode shape, integers under scales of 128
        dict(name="gemv_token", op="gemv", tokens=1, rows=7168, cols=18432, format="int4", group=128, zeros=False),
        # five drafted tokens, an odd number of rows, groups of 32 with zero points
        dict(name="gemv_zeros", op="gemv", tokens=5, rows=4099, cols=7168, format="int4", group=32, zeros=True),
        # 16 sequences through a wide product in e2m1
        dict(name="gemv_wide", op="gemv", tokens=16, rows=18432, cols=7168, format="e2m1", group=32, zeros=False),
        # 33 sequences, groups of 64
        dict(name="gemv_batch", op="gemv", tokens=33, rows=4096, cols=7168, format="int4", group=64, zeros=False),
        # a full decode batch through the experts' down shape
        dict(name="gemv_full", op="gemv", tokens=64, rows=7168, cols=2048, format="int4", group=128, zeros=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        tokens, topk = _log(rng, 1, 64), rng.randint(1, 8)
        ranks = rng.choice([1, 2, 4]) if tokens * topk >= 32 else 1
        return dict(op="moe", tokens=tokens, experts=rng.randint(8, 32), ranks=ranks, topk=topk,
                    hidden=128 * _log(rng, 4, 56), half=128 * _log(rng, 1, 16),
                    weights=rng.choice(["plain", "preshuffled", "w4"]), base=rng.random() < 0.5)
    fmt = rng.choice(["int4", "int4", "e2m1"])
    cols = 128 * _log(rng, 2, 144)
    return dict(op="gemv", tokens=_log(rng, 1, 64), rows=_log(rng, 64, 7168 * 18432 // cols if cols > 7168 else 18432),
                cols=cols, format=fmt, group=32 if fmt == "e2m1" else rng.choice([32, 64, 128]),
                zeros=fmt == "int4" and rng.random() < 0.5)


# ---------------------------------------------------------------- layouts

#: values of the sixteen codes of e2m1
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
#: steps between their magnitudes
STEPS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


def _nibbles(codes):
    """Row-order codes [..., K / 2] (even column in the low half of a byte) -> [..., K]."""
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def _bytes(nibbles):
    return nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)


def _tiles(t, rows=16):
    """[..., N, X] -> [..., ceil(N / rows), rows, X], rows past N zero."""
    pad = -t.shape[-2] % rows
    if pad:
        t = torch.cat([t, t.new_zeros(*t.shape[:-2], pad, t.shape[-1])], -2)
    return t.unflatten(-2, (-1, rows))


def _units(t, n):
    """Columns in units of n, those past the end zero: [..., X] -> [..., ceil(X / n), n]."""
    pad = -t.shape[-1] % n
    if pad:
        t = torch.cat([t, t.new_zeros(*t.shape[:-1], pad)], -1)
    return t.unflatten(-1, (-1, n))


def _shuffled_e4m3(w):
    """fp8_weight_preshuffle's order: [.., 32-row group, K-block, 4 pieces of 1 KB, (half, row), 16 bytes]."""
    E, N, K = w.shape
    v = w.view(E, N // 32, 32, K // 128, 2, 2, 2, 16)  # column = 64 a + 32 half + 16 b + byte
    return v.permute(0, 1, 3, 4, 6, 5, 2, 7).contiguous().view(E, N, K)


def _shuffled_e2m1(codes, scales):
    """w4_preshuffle's order for e2m1: tiles of 16 rows by 128 columns, lane (c, r) holds row r, columns 32 c .. 32 c + 31;
    scales in units of 512 columns, lane (c, r) holds those of its four tiles."""
    c = _tiles(codes).unflatten(-1, (-1, 4, 16)).movedim(-4, -2)  # [.., tile, KB, 4, 16 rows, 16 bytes]
    s = _units(_tiles(scales), 16).unflatten(-1, (4, 4))  # [.., tile, row, unit, block, c]
    n = s.dim()
    s = s.permute(*range(n - 4), n - 3, n - 1, n - 4, n - 2)
    return c.flatten(-3).contiguous(), s.flatten(-3, -2).contiguous()


def _shuffled_int4(codes, scales, zeros):
    """w4_preshuffle's order for integers: in a tile of 16 rows by 128 columns word i of lane (c, r) holds columns
    32 i + 8 c + 0, 2, 4, 6, 1, 3, 5, 7; scales (and zero points) in units of 512 columns."""
    v = _tiles(_nibbles(codes)).unflatten(-1, (-1, 4, 4, 8))[..., [0, 2, 4, 6, 1, 3, 5, 7]]  # [tile, r, KB, i, c, 8]
    c = _bytes(v.permute(0, 2, 4, 1, 3, 5)).flatten(-4).contiguous()
    per = 512 * scales.shape[-1] // (2 * codes.shape[-1])
    s, z = (None if t is None else _units(_tiles(t), per).movedim(-3, -2).contiguous() for t in (scales, zeros))
    return c, s, z


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _quant(v):
    """1x128 groups along the last dimension: (e4m3 codes, UE8M0 bytes [..., groups]); the exponent is the smallest
    with 448 * 2^e >= the group's largest magnitude, at least -42."""
    grouped = v.unflatten(-1, (-1, 128))
    m, x = torch.frexp(grouped.abs().amax(-1))
    e = torch.where(m > 0, x - 9 + (m > 0.875), -42).clamp(min=-42)
    codes = (grouped * torch.exp2(-e.float()).unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2)
    return codes, (e + 127).to(torch.uint8)


def _e2m1_codes(v):
    """Normal values -> row-order codes of e2m1, about as a group's scale leaves them."""
    a = v.abs()
    code = (v < 0).to(torch.uint8) << 3
    for step in STEPS:
        code += a > step
    return _bytes(code)


def _experts(g, s, name, E, N, K, kind):
    """One product's weights: codes of normal values and scales about 2^-12 (e4m3) or 2^-7 (e2m1), in row order and, if
    the case says so, in the library's order (`name` and `s` + `name`, or with a leading underscore)."""
    if kind == "w4":
        codes = torch.stack([_e2m1_codes(torch.randn(N, K, generator=g, device=DEV) * 1.7) for _ in range(E)])
        scales = torch.randint(118, 122, (E, N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
        s[name], s["s" + name] = codes, scales
        s["_" + name], s["_s" + name] = _shuffled_e2m1(codes, scales)
        return
    codes = torch.stack([(torch.randn(N, K, generator=g, device=DEV) * 90).clamp(-448, 448).to(torch.float8_e4m3fn)
                         for _ in range(E)])
    s[name] = codes.view(torch.uint8)
    s["s" + name] = torch.exp2(torch.randint(-13, -10, (E, N // 128, K // 128), generator=g, device=DEV).float())
    s["_" + name] = _shuffled_e4m3(s[name]) if kind == "preshuffled" else s[name]
    s["_s" + name] = s["s" + name]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    T = case["tokens"]
    if case["op"] == "moe":
        E, k, K, H = case["experts"], case["topk"], case["hidden"], case["half"]
        x = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16)
        codes, b = _quant(x.float())
        s["q"] = codes.view(torch.uint8)
        # packed scale words [ceil(K / 512), round_up(T, 4)]: four groups of a row to a word
        b = torch.cat([b, b.new_zeros(-T % 4, b.shape[1])])
        s["sf"] = _units(b, 4).contiguous().view(torch.int32).squeeze(-1).t().contiguous()
        pop = torch.randn(E * case["ranks"], generator=g, device=DEV) * 0.2
        noise = -torch.log(-torch.log(torch.rand(T, E * case["ranks"], generator=g, device=DEV).clamp(1e-7, 1 - 1e-6)))
        ids = (pop + noise).topk(k, dim=1).indices
        s["ids"] = torch.where(ids < E, ids, -1).int()
        w = torch.rand(T, k, generator=g, device=DEV) + 0.1
        s["w"] = w / w.sum(1, keepdim=True)
        s["base"] = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16) if case["base"] else None
        _experts(g, s, "w13", E, 2 * H, K, case["weights"])
        _experts(g, s, "w2", E, K, H, case["weights"])
        return s
    N, K, G = case["rows"], case["cols"], case["group"]
    x = torch.randn(T, K, generator=g, device=DEV)
    # one entry in a hundred is an outlier, as activations have them
    s["x"] = torch.where(torch.rand(T, K, generator=g, device=DEV) < 0.01, x * 50, x).to(torch.bfloat16)
    s["z"] = s["_z"] = None
    v = torch.randn(N, K, generator=g, device=DEV)
    if case["format"] == "e2m1":
        s["c"] = _e2m1_codes(v * 1.7)
        s["s"] = torch.randint(118, 122, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
        s["_c"], s["_s"] = _shuffled_e2m1(s["c"], s["s"])
        return s
    if case["zeros"]:
        s["z"] = torch.randint(5, 12, (N, K // G), generator=g, device=DEV, dtype=torch.uint8)
    mid = 8 if s["z"] is None else s["z"].repeat_interleave(G, 1).float()
    s["c"] = _bytes((torch.round(v * 2.5) + mid).clamp(0, 15).to(torch.uint8))
    s["s"] = ((torch.rand(N, K // G, generator=g, device=DEV) + 0.5) * 0.008).to(torch.bfloat16)
    s["_c"], s["_s"], s["_z"] = _shuffled_int4(s["c"], s["s"], s["z"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _values(s, name, at=None):
    """A product's weights in 32 bits, of all experts or of those at `at`."""
    c, f = (s[name], s["s" + name]) if at is None else (s[name][at], s["s" + name][at])
    if s["weights"] == "w4":
        v = torch.tensor(E2M1, device=c.device)[_nibbles(c).int()]
        return (v.unflatten(-1, (-1, 32)) * torch.exp2(f.float() - 127).unsqueeze(-1)).flatten(-2)
    E, N, K = c.shape
    v = c.view(torch.float8_e4m3fn).float().view(E, N // 128, 128, K // 128, 128)
    return (v * f.view(E, N // 128, 1, K // 128, 1)).view(E, N, K)


def _plain_moe(s):
    T, K, k = s["tokens"], s["hidden"], s["topk"]
    b = s["sf"].t()[:T].contiguous().view(torch.uint8)[:, : K // 128]
    x = (s["q"].view(torch.float8_e4m3fn).float().view(T, -1, 128) * torch.exp2(b.float() - 127).unsqueeze(-1)).view(T, K)
    some, ids = s["ids"] >= 0, s["ids"].clamp(min=0).long()
    few = T * k <= s["experts"]  # the pairs' experts, or all of them
    at = ids.flatten() if few else None
    rows = x.repeat_interleave(k, 0).unsqueeze(1) if few else x.unsqueeze(0)
    gate, up = torch.matmul(rows, _values(s, "w13", at).transpose(1, 2)).chunk(2, -1)
    codes, b = _quant(gate / (1 + torch.exp(-gate)) * up)
    y = (codes.float().unflatten(-1, (-1, 128)) * torch.exp2(b.float() - 127).unsqueeze(-1)).flatten(-2)
    y = torch.matmul(y, _values(s, "w2", at).transpose(1, 2))
    y = y.view(T, k, K) if few else y[ids, torch.arange(T, device=ids.device).unsqueeze(1)]
    out = torch.where(some.unsqueeze(-1), s["w"].unsqueeze(-1) * y, 0).sum(1)
    return (out if s["base"] is None else s["base"].float() + out).to(torch.bfloat16)


def _own_moe(s):
    import block_scaled_fp8_token_amd as F
    call = {"plain": F.moe_decode_layer, "preshuffled": F.moe_decode_layer_preshuffled, "w4": F.moe_decode_layer_w4}
    return call[s["weights"]](s["q"], s["sf"], s["ids"], s["w"], s["_w13"], s["_sw13"], s["_w2"], s["_sw2"],
                              base=s["base"])


def _plain_gemv(s):
    c = _nibbles(s["c"])
    if s["format"] == "e2m1":
        w = torch.tensor(E2M1, device=c.device)[c.int()].unflatten(-1, (-1, 32))
        w = w * torch.exp2(s["s"].float() - 127).unsqueeze(-1)
    else:
        z = 8 if s["z"] is None else s["z"].float().unsqueeze(-1)
        w = (c.float().unflatten(-1, (-1, s["group"])) - z) * s["s"].float().unsqueeze(-1)
    return torch.matmul(s["x"].float(), w.flatten(-2).t()).to(torch.bfloat16)


def _own_gemv(s):
    import block_scaled_fp8_token_amd as F
    return F.w4_group_gemv_nt(s["x"], s["_c"], s["_s"], s["rows"], zeros=s["_z"])


_plain = {"moe": _plain_moe, "gemv": _plain_gemv}
_own = {"moe": _own_moe, "gemv": _own_gemv}


# ---------------------------------------------------------------- what a pass has to do

def work(case):
    T = case["tokens"]
    if case["op"] == "moe":
        E, k, K, H = case["experts"], case["topk"], case["hidden"], case["half"]
        pairs = T * k / case["ranks"]
        read = E * (1 - (1 - k / (E * case["ranks"])) ** T)  # experts that some token has chosen, as expected
        each = 3 * H * K
        weights = each / 2 + each / 32 if case["weights"] == "w4" else each + 4 * each / 16384
        rows = T * (K + K // 128 + 2 * K + (2 * K if case["base"] else 0) + 8 * k)
        return {"bytes": read * weights + rows, "flops": 2 * pairs * each}
    N, K, G = case["rows"], case["cols"], case["group"]
    scales = 1 if case["format"] == "e2m1" else 3 if case["zeros"] else 2
    return {"bytes": N * K / 2 + scales * N * K / G + 2 * T * (N + K), "flops": 2 * T * N * K}


# ---------------------------------------------------------------- the same in 64 bits

def _rounded_e4m3(v):
    """v (at most 448) to the nearest value of e4m3, ties to the even one."""
    step = torch.exp2(torch.frexp(v).exponent.clamp(min=-5).double() - 4)
    return torch.round(v / step) * step


def _grouped_e4m3(v):
    """The values that v's 1x128 groups stand for once they are in e4m3 under their power of two."""
    v = v.view(-1, v.shape[-1] // 128, 128)
    most = v.abs().amax(-1, keepdim=True).clamp(min=1e-10) / 448
    up = torch.exp2(torch.ceil(torch.log2(most)))
    up = torch.where(up / 2 >= most, up / 2, torch.where(up < most, up * 2, up))  # log2 is off by an ulp at powers of two
    return (_rounded_e4m3(v / up) * up).flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    T = case["tokens"]
    pow2 = lambda b: torch.exp2(b.double() - 127)  # noqa: E731
    table = torch.tensor(E2M1, dtype=torch.float64, device=DEV)

    def four(c):
        out = torch.empty(*c.shape[:-1], 2 * c.shape[-1], dtype=torch.uint8, device=DEV)
        out[..., 0::2] = c % 16
        out[..., 1::2] = c // 16
        return out

    if case["op"] == "gemv":
        c, G = four(s["c"]), case["group"]
        wide = lambda t: t.repeat_interleave(G, dim=1)  # noqa: E731
        if case["format"] == "e2m1":
            w = table[c.int()] * wide(pow2(s["s"]))
        else:
            w = (c.double() - (8 if s["z"] is None else wide(s["z"].double()))) * wide(s["s"].double())
        return s["x"].double() @ w.t()
    K, H = case["hidden"], case["half"]
    words = s["sf"].cpu().numpy().view("uint32")
    b = torch.tensor([[int(words[g // 4, t]) >> 8 * (g % 4) & 255 for g in range(K // 128)] for t in range(T)], device=DEV)
    x = s["q"].view(torch.float8_e4m3fn).double() * pow2(b).repeat_interleave(128, dim=1)
    out = torch.zeros(T, K, dtype=torch.float64, device=DEV) if s["base"] is None else s["base"].double()

    def weights(name, e):
        c, f = s[name][e], s["s" + name][e]
        if case["weights"] == "w4":
            return table[four(c).int()] * pow2(f).repeat_interleave(32, dim=1)
        f = f.double().repeat_interleave(128, dim=0).repeat_interleave(128, dim=1)
        return c.view(torch.float8_e4m3fn).double() * f

    for e in range(case["experts"]):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel():
            h = x[t] @ weights("w13", e).t()
            y = _grouped_e4m3(h[:, :H] * torch.sigmoid(h[:, :H]) * h[:, H:])
            out.index_add_(0, t, s["w"][t, j].double().unsqueeze(1) * (y @ weights("w2", e).t()))
    return out
