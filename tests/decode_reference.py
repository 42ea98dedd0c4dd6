"""Plain references in 64 bits of the operators of a decode step (not a test module): written
from the formulas and layouts of include/fp8bs.h, on the CPU, without the library."""
from __future__ import annotations

import numpy as np
import torch

F32_U = 2.0 ** -24  # unit roundoff of fp32
BF16_U = 2.0 ** -8  # and of bf16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def nibbles(codes):
    """codes [..., K/2], the even column in the low half of a byte -> [..., K]."""
    out = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]), np.uint8)
    out[..., 0::2] = codes & 15
    out[..., 1::2] = codes >> 4
    return out


def packed(n):
    n = n.astype(np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def bf16_values(t):
    """A bf16 tensor's values (numpy has no such type)."""
    return t.detach().cpu().double().numpy()


def w4_values(codes, scales, zeros=None):
    """Row-order 4-bit weights [..., N, K]: uint8 scales are UE8M0 bytes of e2m1, float ones the scales of integers."""
    n = nibbles(codes)
    group = n.shape[-1] // scales.shape[-1]

    def wide(v):
        return np.repeat(v.astype(np.float64), group, -1)
    if scales.dtype == np.uint8:
        return E2M1[n] * np.exp2(wide(scales) - 127)
    return (n - (8.0 if zeros is None else wide(zeros))) * wide(scales)


def round_bf16(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16)


def quant_e2m1(w):
    """w [N, K] fp64 holding bf16 values -> codes (nibbles), UE8M0 bytes."""
    g = w.reshape(w.shape[0], -1, 32)
    most = np.abs(g).max(-1)
    m, x = np.frexp(most)  # most = m 2^x, m in [0.5, 1): 6 2^e >= most where m 2^(x - 3) <= 0.75
    e = np.where(most > 0, x - 3 + (m > 0.75), -126)
    e = np.maximum(e, -126)
    v = np.abs(g) / np.exp2(e)[..., None]
    mags = E2M1[:8]
    code = np.zeros(v.shape, np.int64)
    for i in range(7):  # to the nearest, a tie to the even code
        mid = (mags[i] + mags[i + 1]) / 2
        code = np.where((v > mid) | ((v == mid) & (i % 2 == 1)), i + 1, code)
    code = code + 8 * np.signbit(g)
    return code.reshape(w.shape), (e + 127).astype(np.uint8)


def quant_int4(w, group, zero_points):
    """w [N, K] fp32 holding bf16 values -> codes (nibbles), bf16 scales (a tensor), zero points; in fp32 as stated."""
    f = np.float32
    g = w.astype(f).reshape(w.shape[0], -1, group)
    lo, hi = np.minimum(g.min(-1), f(0)), np.maximum(g.max(-1), f(0))
    s = round_bf16((hi - lo) / f(15) if zero_points else np.maximum(-lo, hi) / f(7))
    sv = s.float().numpy()
    some = sv > 0
    div = np.where(some, sv, f(1))
    z = np.minimum(np.rint(-lo / div), f(15)) if zero_points else np.full(sv.shape, f(8))
    z = np.where(some, z, f(0) if zero_points else f(8)).astype(f)
    c = np.clip(np.rint(g / div[..., None]) + z[..., None], 0, 15)
    c = np.where(some[..., None], c, z[..., None])
    return c.reshape(w.shape).astype(np.int64), s, z.astype(np.uint8)


def preshuffled(codes, scales, zeros=None):
    """w4_preshuffle of [N, K/2] codes, entry by entry: (codes [tiles, KB, 1024], scales, zeros)."""
    N, half = codes.shape
    K = 2 * half
    KB, tiles, units = K // 128, -(-N // 16), -(-K // 512)
    e2m1 = scales.dtype == np.uint8
    n = np.zeros((tiles * 16, K), np.uint8)
    n[:N] = nibbles(codes)
    lanes = np.zeros((tiles, KB, 64, 32), np.uint8)
    for lane in range(64):
        c, r = divmod(lane, 16)
        rows = n[r::16]
        for kb in range(KB):
            if e2m1:
                cols = 128 * kb + 32 * c + np.arange(32)
            else:
                cols = np.concatenate([128 * kb + 32 * i + 8 * c + np.array([0, 2, 4, 6, 1, 3, 5, 7]) for i in range(4)])
            lanes[:, kb, lane] = rows[:, cols]
    out = packed(lanes).reshape(tiles, KB, 1024)

    def units_of(v):
        groups = v.shape[1]
        per = 512 * groups // K
        padded = np.zeros((tiles * 16, units * per), v.dtype)
        padded[:N, :groups] = v
        padded = padded.reshape(tiles, 16, units, per)
        if not e2m1:
            return padded.transpose(0, 2, 1, 3).copy()
        s = np.zeros((tiles, units, 64, 4), v.dtype)
        for lane in range(64):
            c, r = divmod(lane, 16)
            for b in range(4):
                s[:, :, lane, b] = padded[:, r, :, 4 * b + c]
        return s
    return out, units_of(scales), None if zeros is None else units_of(zeros)


def e4m3_step(v):
    """Distance of neighbouring e4m3 values at |v| (2^-9 under the smallest normal one)."""
    _, x = np.frexp(np.abs(v))
    return np.exp2(np.maximum(x, -5) - 4.0)


def quant_group(y, dy):
    """1x128 groups of y [..., H] to e4m3 under a power of two, as values, and how far each may be from the value of
    a y that is off by at most dy: nothing where no decision is near, else what the other choice changes."""
    g, d = y.reshape(*y.shape[:-1], -1, 128), dy.reshape(*y.shape[:-1], -1, 128)

    def exponent(most):
        m, x = np.frexp(np.maximum(most, 1e-10))
        return np.maximum(x - 9 + (m > 0.875), -42)

    def at(e):
        s = np.exp2(e)[..., None]
        step = e4m3_step(g / s) * s
        q = np.round(g / step) * step
        near = np.abs(np.abs(g / step - np.floor(g / step)) - 0.5) * step <= d
        return q, np.where(near, step, 0.0)
    most = np.abs(g).max(-1)
    slack = d.max(-1)
    e, lo, hi = exponent(most), exponent(np.maximum(most - slack, 0)), exponent(most + slack)
    q, off = at(e)
    for other in (lo, hi):  # a largest magnitude next to a border: the other scale's values too
        q2, off2 = at(other)
        off = np.maximum(off, np.abs(q2 - q) + off2)
    return q.reshape(y.shape), off.reshape(y.shape)


def moe_layer(x, ids, weights, w13, w2, base=None):
    """x [T, K] values, ids and weights [T, k], w13 [E, 2H, K], w2 [E, K, H] values, base [T, K] or None ->
    (out fp64 [T, K], how far a bf16 result with fp32 sums may be)."""
    T, K = x.shape
    E, H = w13.shape[0], w2.shape[2]
    out = np.zeros((T, K)) if base is None else np.array(base, np.float64)
    size = np.abs(out)
    off = np.zeros((T, K))
    # a product over K in fp32: 32 columns a matrix instruction, K / 32 of them in turn, 16 wavefronts' sums; each addition
    # is off by at most 2^-24 of what was summed (and again that where the instruction cuts off instead of rounding)
    g_dot, g_out = (2 * (32 + n / 32 + 16) * F32_U for n in (K, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        h, a = x[t] @ w13[e].T, np.abs(x[t]) @ np.abs(w13[e]).T * g_dot
        gate, up = h[:, :H], h[:, H:]
        with np.errstate(over="ignore"):
            silu = gate / (1 + np.exp(-gate))
        y = silu * up
        # |silu'| <= 1.1; the exponential, division and product are off by a few ulps
        q, dq = quant_group(y, 1.1 * np.abs(up) * a[:, :H] + np.abs(silu) * a[:, H:] + 16 * F32_U * np.abs(y) + 1e-40)
        w = weights[t, j][:, None].astype(np.float64)
        np.add.at(out, t, w * (q @ w2[e].T))
        part = np.abs(w) * (np.abs(q) @ np.abs(w2[e]).T)
        np.add.at(size, t, part)
        np.add.at(off, t, np.abs(w) * (dq @ np.abs(w2[e]).T) + g_out * part)
    return out, off + 64 * F32_U * size + BF16_U * (np.abs(out) + off)
