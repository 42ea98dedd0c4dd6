"""Plain references in 64 bits of the operators around the experts' products (not a test
module): written from the formulas of include/fp8bs.h, on the CPU, without the library."""
from __future__ import annotations

import math

import numpy as np

F32_U = 2.0 ** -24  # unit roundoff of fp32
BF16_U = 2.0 ** -8  # and of bf16 (8 significant bits)


def sigmoid(v):
    v = np.asarray(v, np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def softmax(v):
    """Over the last axis; -inf has no share; a row of nothing but -inf is zero."""
    m = v.max(-1, keepdims=True)
    e = np.exp(v - np.where(np.isfinite(m), m, 0.0))
    z = e.sum(-1, keepdims=True)
    return np.divide(e, z, out=np.zeros_like(e), where=z > 0)


def route(logits, topk, bias=None, groups=1, topk_groups=1, group_top=1, scoring="softmax", renormalize=True,
          scale=1.0):
    """(ids, weights, gap): gap is the smallest distance between two different numbers that the
    choice compares, so that a caller can see that fp32 orders them alike."""
    T, E = logits.shape
    ids = np.full((T, topk), -1, np.int64)
    w = np.zeros((T, topk))
    gap = math.inf

    def note(values):
        nonlocal gap
        v = np.unique(values[np.isfinite(values)])
        if v.size > 1:
            gap = min(gap, float(np.diff(v).min()))

    for t in range(T):
        l = logits[t].astype(np.float64)
        l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
        s = sigmoid(l) if scoring == "sigmoid" else softmax(l)
        ok = l > -np.inf
        if bias is None:
            rank = l.copy()
        else:
            rank = np.where(ok, s + bias, -np.inf)
            rank = np.where(rank > -np.inf, rank, -np.inf)
        if groups > 1:
            size = E // groups
            score = np.full(groups, -np.inf)
            for g in range(groups):
                part = rank[g * size:(g + 1) * size]
                if group_top == 2 and bias is None:
                    part = np.where(part > -np.inf, s[g * size:(g + 1) * size], -np.inf)
                best = np.sort(part)[::-1][:group_top]
                best = best[best > -np.inf]
                if best.size:
                    score[g] = best.sum()
            note(score)
            kept = np.argsort(-score, kind="stable")[:topk_groups]
            keep = np.zeros(groups, bool)
            keep[kept] = True
            rank = np.where(np.repeat(keep, size), rank, -np.inf)
        note(rank)
        order = np.argsort(-rank, kind="stable")[:topk]
        order = order[rank[order] > -np.inf]
        n = order.size
        ids[t, :n] = order
        c = s[order]
        if renormalize and n:
            c = softmax(l[order]) if scoring == "softmax" else (c / c.sum() if c.sum() > 0 else 0 * c)
        w[t, :n] = scale * c
    return ids, w, gap


def route_weights(l, ids, scoring, renormalize, scale):
    """Weights of chosen experts as a function of the logits [T, E], for differences (all ids valid)."""
    s = sigmoid(l) if scoring == "sigmoid" else softmax(l)
    c = np.take_along_axis(s, ids, 1)
    return scale * (c / c.sum(1, keepdims=True) if renormalize else c)


def combine(y, ids, slots, weights, base):
    """(out, sum of magnitudes): y [E, M, N], ids and slots [T, k]."""
    E, M, N = y.shape
    T, k = ids.shape
    out = np.zeros((T, N)) if base is None else base.astype(np.float64).copy()
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            e, s = ids[t, j], slots[t, j]
            if 0 <= e < E and 0 <= s < M:
                v = (1.0 if weights is None else float(weights[t, j])) * y[e, s].astype(np.float64)
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


def rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def norm(x, w_pre, y=None, w_post=None, gate=None, residual_scale=1.0, eps=1e-6, offset=0.0):
    h = residual_scale * x.astype(np.float64)
    if y is not None:
        b = y.astype(np.float64)
        if w_post is not None:
            b = b * rms(b, eps) * (w_post.astype(np.float64) + offset)
        if gate is not None:
            b = b * gate.astype(np.float64)
        h = h + b
    return h, h * rms(h, eps) * (w_pre.astype(np.float64) + offset)


def e4m3_decode(codes):
    codes = np.asarray(codes, np.uint8).astype(np.int64)
    sign = np.where(codes & 0x80, -1.0, 1.0)
    exp, man = (codes >> 3) & 15, codes & 7
    return sign * np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp - 10.0))


def scale_bytes(words, rows, groups):
    """UE8M0 bytes [rows, groups] of packed words uint32 [W, >= rows]."""
    w = np.asarray(words).view(np.uint32)[:, :rows]
    b = np.stack([(w >> (8 * i)) & 0xFF for i in range(4)], -1)  # [W, rows, 4]
    b = b.transpose(1, 0, 2).reshape(rows, -1)
    assert (b[:, groups:] == 0).all(), "bytes past the row's groups are zero"
    return b[:, :groups]


def check_quantized(ref, codes, words, err):
    """codes [rows, K] and packed words quantize values within err (an array, or a number) of ref (64
    bits): every exponent is the smallest e with 448 * 2^e >= max(amax, 1e-10), and every decoded value
    is the nearest of the e4m3 grid."""
    rows, K = ref.shape
    G = K // 128
    err = np.broadcast_to(np.asarray(err, np.float64), ref.shape)
    e = scale_bytes(words, rows, G).astype(np.int64) - 127
    s = 2.0 ** e
    lo = np.maximum(np.abs(ref) - err, 0).reshape(rows, G, 128).max(-1)
    hi = (np.abs(ref) + err).reshape(rows, G, 128).max(-1)
    assert (np.maximum(lo, 1e-10) <= 448 * s).all(), "a scale is too small"
    assert ((np.maximum(hi, 1e-10) > 224 * s) | (e == -42)).all(), "a scale is too large"
    s = np.repeat(s, 128, 1)
    got = e4m3_decode(codes) * s
    # grid step at the largest magnitude the value can have: 2^-3 of its binade, 2^-9 of the scale at least
    top = np.maximum((np.abs(ref) + err) / s, 2.0 ** -60)
    step = np.maximum(2.0 ** (np.floor(np.log2(top)) - 3), 2.0 ** -9) * s
    bad = ~(np.abs(got - ref) <= (step / 2 + err) * (1 + 1e-12))
    assert not bad.any(), "%d of %d codes off, first at %s" % (bad.sum(), bad.size, np.argwhere(bad)[:3].tolist())
