"""The operators around the experts' products: routing, combine, the norms of the residual
stream, and the 8-bit checkpoint of the gated activation, each with its backward pass.

Binding of the entry points of the same names in include/fp8bs.h (which states the
formulas).  Wrong types, shapes and strides raise TypeError or ValueError before
anything is launched; all tensors of a call lie on the current device.

The calls take tensors for their values: as everywhere in this binding, nothing is recorded for
automatic differentiation and results do not require a gradient, whatever the inputs say.  A
training step calls the backward entry points itself, or wraps a pair of calls in a
torch.autograd.Function.  Outputs that a caller passes must not overlap inputs (not checked).
"""
from __future__ import annotations

import torch

from . import _check, _lib, _words

__all__ = [
    "moe_route_topk", "moe_route_topk_backward", "moe_combine", "moe_combine_backward", "residual_rms_norm",
    "residual_rms_norm_backward", "silu_mul_quant_group_pack_checkpoint", "silu_mul_backward_from_checkpoint",
]

_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_U32 = (torch.int32, torch.uint32)
_E4M3 = (torch.uint8, torch.float8_e4m3fn, torch.int8)
_FLOAT = (torch.bfloat16, torch.float32)
_SCORING = {"sigmoid": 0, "softmax": 1}
_OUT = {"bf16": (True, False), "fp8": (False, True), "both": (True, True)}


def _typed(t, name, dtypes):
    if t.dtype not in dtypes:
        raise TypeError("%s: dtype %s not in %s" % (name, t.dtype, dtypes))


def _whole(t, name, dtypes, shape):
    """A contiguous tensor of that shape; its address."""
    if t.dtype not in dtypes:
        _typed(t, name, dtypes)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous %s, got shape %s strides %s"
                         % (name, list(shape), list(t.shape), list(t.stride())))
    return t.data_ptr()


def _rows(t, name, dtypes, rows, cols):
    """A 2-D [rows, cols] tensor with unit column stride; its address and row stride."""
    if t.dtype not in dtypes:
        _typed(t, name, dtypes)
    if t.shape != (rows, cols):
        raise ValueError("%s must be %s, got %s" % (name, [rows, cols], list(t.shape)))
    ld, unit = t.stride()
    if rows <= 1:
        ld = cols  # the stride of a single row means nothing
    if (unit != 1 and cols > 1) or ld < cols:
        raise ValueError("%s must have unit column stride and row stride >= %d, got strides %s"
                         % (name, cols, list(t.stride())))
    return t.data_ptr(), ld


def _beside(t, name, like):
    if t.get_device() != like.get_device():
        raise ValueError("%s: every tensor must be a device tensor, all on one device" % name)


def _out(t, name, dtypes, shape, like):
    """An output the caller may have passed, or a new one of dtypes[0] beside `like`; its address."""
    if t is None:
        t = like.new_empty(shape, dtype=dtypes[0])
        return t, t.data_ptr()
    _beside(t, name, like)
    return t, _whole(t, name, dtypes, shape)


def _out_rows(t, name, dtypes, rows, cols, like):
    """The same of a 2-D output that may be strided; its address and row stride."""
    if t is None:
        t = like.new_empty((rows, cols), dtype=dtypes[0])
        return t, t.data_ptr(), cols
    _beside(t, name, like)
    return t, *_rows(t, name, dtypes, rows, cols)


def _2d(t, name):
    if t.dim() != 2:
        raise ValueError("%s must have 2 dims, got %d" % (name, t.dim()))
    return t.shape


# The raw handle of the current stream: building a Stream object for it costs 2.7 us on the
# measured host, which a single-token call would notice.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _on_stream(stream, fn, *args):
    """fn(*args) on a stream that the caller names: new outputs come from that stream's memory, and
    the tensors that the caller passed are kept until its work on them is done."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    if stream == torch.cuda.current_stream():
        return fn(*args)
    with torch.cuda.stream(stream):
        got = fn(*args)
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return got


def _launch(name, inputs, *args):
    """Calls the library on the current stream once every input is known to lie on the current
    device (the outputs lie beside an input, see _out)."""
    dev = inputs[0].get_device()
    for t in inputs:
        if t is not None and t.get_device() != dev:
            dev = -1
    if dev < 0:
        raise ValueError("%s: every tensor must be a device tensor, all on one device" % name)
    if dev != _current_device():
        raise ValueError("%s: the tensors are on cuda:%d, which is not the current device" % (name, dev))
    st = getattr(_lib, name)(*args, _raw_stream(dev))
    if st:
        _check(name, st)


def moe_route_topk(logits: torch.Tensor, topk: int, bias: torch.Tensor | None = None, groups: int = 1,
                   topk_groups: int = 1, group_top: int = 1, scoring: str = "softmax", renormalize: bool = True,
                   scale: float = 1.0, topk_ids: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                   stream=None):
    """Choose topk of E experts per token.  logits fp32 or bf16 [T, E] -> (topk_ids int32 [T, topk],
    weights fp32 [T, topk]).  scoring "sigmoid" or "softmax"; bias fp32 [E] is added to the scores for the
    choice only; groups > 1 restricts the choice to the topk_groups groups of the best score (their best rank,
    or with group_top = 2 the sum of the two best).  Experts with a logit of -inf or NaN are not available;
    ids that are left over are -1 with weight 0."""
    if stream is not None:
        return _on_stream(stream, moe_route_topk, logits, topk, bias, groups, topk_groups, group_top, scoring,
                          renormalize, scale, topk_ids, weights)
    T, E = _2d(logits, "logits")
    pl, ld = _rows(logits, "logits", _FLOAT, T, E)
    if scoring not in _SCORING:
        raise ValueError("scoring must be 'sigmoid' or 'softmax', got %r" % (scoring,))
    pb = None if bias is None else _whole(bias, "bias", _F32, (E,))
    topk_ids, pi = _out(topk_ids, "topk_ids", _I32, (T, topk), logits)
    weights, pw = _out(weights, "weights", _F32, (T, topk), logits)
    _launch("moe_route_topk", (logits, bias), pl, logits.dtype == torch.float32, ld, T, E, pb,
            _SCORING[scoring], groups, topk_groups, group_top, topk, bool(renormalize), scale, pi, pw)
    return topk_ids, weights


def moe_route_topk_backward(logits: torch.Tensor, topk_ids: torch.Tensor, d_weights: torch.Tensor,
                            scoring: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                            d_logits: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of moe_route_topk's weights with respect to the logits, the choice held fixed: d_weights fp32
    [T, topk] -> d_logits [T, E] of the logits' type.  scoring, renormalize and scale are the forward's."""
    if stream is not None:
        return _on_stream(stream, moe_route_topk_backward, logits, topk_ids, d_weights, scoring, renormalize, scale,
                          d_logits)
    T, E = _2d(logits, "logits")
    pl, ld = _rows(logits, "logits", _FLOAT, T, E)
    topk = _2d(topk_ids, "topk_ids")[1]
    if scoring not in _SCORING:
        raise ValueError("scoring must be 'sigmoid' or 'softmax', got %r" % (scoring,))
    pi = _whole(topk_ids, "topk_ids", _I32, (T, topk))
    pw = _whole(d_weights, "d_weights", _F32, (T, topk))
    d_logits, pd, ld_d = _out_rows(d_logits, "d_logits", (logits.dtype,), T, E, logits)
    _launch("moe_route_topk_backward", (logits, topk_ids, d_weights), pl,
            logits.dtype == torch.float32, ld, T, E, pi, pw, _SCORING[scoring], topk, bool(renormalize), scale, pd, ld_d)
    return d_logits


def moe_combine(y: torch.Tensor, topk_ids: torch.Tensor, slot_of: torch.Tensor, weights: torch.Tensor | None = None,
                base: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Experts' rows back to their tokens: out[t] = base[t] + sum_j weights[t, j] * y[topk_ids[t, j], slot_of[t, j]].
    y bf16 [E, M_max, N], topk_ids and slot_of int32 [T, topk] (as fp8_quant_group_pack_to_experts gives them; pairs
    without a row are left out), weights fp32 [T, topk] (None: ones), base bf16 [T, N] -> bf16 [T, N]."""
    if stream is not None:
        return _on_stream(stream, moe_combine, y, topk_ids, slot_of, weights, base, out)
    if y.dim() != 3:
        raise ValueError("y must be [E, M_max, N]")
    E, M_max, N = y.shape
    T, topk = _2d(topk_ids, "topk_ids")
    py = _whole(y, "y", _BF16, y.shape)
    pi = _whole(topk_ids, "topk_ids", _I32, (T, topk))
    ps = _whole(slot_of, "slot_of", _I32, (T, topk))
    pw = None if weights is None else _whole(weights, "weights", _F32, (T, topk))
    pb, ld_b = (None, 0) if base is None else _rows(base, "base", _BF16, T, N)
    out, po, ld_o = _out_rows(out, "out", _BF16, T, N, y)
    _launch("moe_combine", (y, topk_ids, slot_of, weights, base), py, pi, ps, pw, pb, ld_b, T, topk, E,
            M_max, N, po, ld_o)
    return out


def moe_combine_backward(d_out: torch.Tensor, y: torch.Tensor, topk_ids: torch.Tensor, slot_of: torch.Tensor,
                         weights: torch.Tensor | None = None, quantize: bool = False, d_y: torch.Tensor | None = None,
                         q: torch.Tensor | None = None, sf: torch.Tensor | None = None,
                         d_weights: torch.Tensor | None = None, stream=None):
    """Gradients of moe_combine for d_out bf16 [T, N]: (d_y bf16 [E, M_max, N], d_weights fp32 [T, topk]), or with
    quantize (q uint8 [E, M_max, N], sf int32 [E, ceil(N/512), M_max], d_weights) in the masked GEMM's layout.
    d_weights is None where weights is.  Rows of no pair are not written.  (d_out is base's gradient as it is.)"""
    if stream is not None:
        return _on_stream(stream, moe_combine_backward, d_out, y, topk_ids, slot_of, weights, quantize, d_y, q, sf,
                          d_weights)
    if y.dim() != 3:
        raise ValueError("y must be [E, M_max, N]")
    E, M_max, N = y.shape
    T, topk = _2d(topk_ids, "topk_ids")
    pd, ld_d = _rows(d_out, "d_out", _BF16, T, N)
    py = _whole(y, "y", _BF16, y.shape)
    pi = _whole(topk_ids, "topk_ids", _I32, (T, topk))
    ps = _whole(slot_of, "slot_of", _I32, (T, topk))
    pw = pdw = None
    if weights is not None:
        pw = _whole(weights, "weights", _F32, (T, topk))
        d_weights, pdw = _out(d_weights, "d_weights", _F32, (T, topk), y)
    elif d_weights is not None:
        raise ValueError("d_weights without weights")
    pdy = pq = psf = None
    if quantize:
        if d_y is not None:
            raise ValueError("d_y is not written with quantize")
        q, pq = _out(q, "q", _E4M3, (E, M_max, N), y)
        sf, psf = _out(sf, "sf", _U32, (E, _words(N), M_max), y)
    else:
        if q is not None or sf is not None:
            raise ValueError("q and sf are written with quantize only")
        d_y, pdy = _out(d_y, "d_y", _BF16, (E, M_max, N), y)
    _launch("moe_combine_backward", (d_out, y, topk_ids, slot_of, weights), pd, ld_d, py,
            pi, ps, pw, T, topk, E, M_max, N, pdy, pq, psf, pdw)
    return (q, sf, d_weights) if quantize else (d_y, d_weights)


def _gate(gate, T, N):
    """Address and row stride of a gate [N] (stride 0) or [T, N]."""
    if gate is None:
        return None, 0
    if gate.dim() == 1:
        return _whole(gate, "gate", _BF16, (N,)), 0
    return _rows(gate, "gate", _BF16, T, N)


def residual_rms_norm(x: torch.Tensor, w_pre: torch.Tensor, y: torch.Tensor | None = None,
                      w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                      residual_scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0, out: str = "bf16",
                      h: torch.Tensor | None = None, z: torch.Tensor | None = None, q: torch.Tensor | None = None,
                      sf: torch.Tensor | None = None, stream=None):
    """The norm after a block (of its output y, with w_post), the block's gate, the scaled residual and the norm
    before the next block in one pass:
        h = residual_scale * x + gate * norm(y, w_post),   z = norm(h, w_pre)
    x bf16 or fp32 [T, N], y bf16 [T, N], w_pre and w_post bf16 [N], gate bf16 [N] or [T, N].  out "bf16": z bf16
    [T, N]; "fp8": q uint8 [T, N] and sf int32 [ceil(N/512), round_up(T, 4)] as fp8_quant_group_pack gives them;
    "both".  Returns (h, z, q, sf), None for what is not asked for.  Without y and with residual_scale 1, h is x itself
    and is not written (pass h to have a copy)."""
    if stream is not None:
        return _on_stream(stream, residual_rms_norm, x, w_pre, y, w_post, gate, residual_scale, eps, weight_offset,
                          out, h, z, q, sf)
    T, N = _2d(x, "x")
    px, ldx = _rows(x, "x", _FLOAT, T, N)
    if out not in _OUT:
        raise ValueError("out must be 'bf16', 'fp8' or 'both', got %r" % (out,))
    want_z, want_q = _OUT[out]
    if y is None and (w_post is not None or gate is not None):
        raise ValueError("w_post and gate apply to y")
    py, ldy = (None, 0) if y is None else _rows(y, "y", _BF16, T, N)
    pwp = None if w_post is None else _whole(w_post, "w_post", _BF16, (N,))
    pw = _whole(w_pre, "w_pre", _BF16, (N,))
    pg, ld_g = _gate(gate, T, N)
    ph, ldh, pz, ldz, pq, ldq, psf, ld_sf = None, 0, None, 0, None, 0, None, 0
    if h is not None or y is not None or residual_scale != 1.0:
        h, ph, ldh = _out_rows(h, "h", (x.dtype,), T, N, x)
    if want_z:
        z, pz, ldz = _out_rows(z, "z", _BF16, T, N, x)
    elif z is not None:
        raise ValueError("z is not written with out=%r" % out)
    if want_q:
        W = _words(N)
        q, pq, ldq = _out_rows(q, "q", _E4M3, T, N, x)
        if sf is None:
            sf = x.new_empty((W, max(4, (T + 3) // 4 * 4)), dtype=torch.int32)
        else:
            _beside(sf, "sf", x)
            _typed(sf, "sf", _U32)
        if sf.dim() != 2 or sf.shape[0] != W or sf.shape[1] < T or sf.stride(1) != 1 or sf.stride(0) < T:
            raise ValueError("sf must be [%d, >= %d] with unit column stride, got shape %s strides %s"
                             % (W, T, list(sf.shape), list(sf.stride())))
        psf, ld_sf = sf.data_ptr(), sf.stride(0)
    elif q is not None or sf is not None:
        raise ValueError("q and sf are not written with out=%r" % out)
    _launch("residual_rms_norm", (x, y, w_post, gate, w_pre), px, ldx, x.dtype == torch.float32, py,
            ldy, pwp, pg, ld_g, pw, residual_scale, eps, weight_offset, T, N, ph, ldh, pz, ldz, pq, ldq, psf, ld_sf)
    return x if h is None else h, z, q, sf


def residual_rms_norm_backward(d_z: torch.Tensor, h: torch.Tensor, w_pre: torch.Tensor,
                               d_h: torch.Tensor | None = None, y: torch.Tensor | None = None,
                               w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                               residual_scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0,
                               d_x: torch.Tensor | None = None, d_y: torch.Tensor | None = None,
                               d_w_pre: torch.Tensor | None = None, d_w_post: torch.Tensor | None = None,
                               d_gate: torch.Tensor | None = None, stream=None):
    """Gradients of residual_rms_norm: from d_z bf16 [T, N], the h it returned and (with the residual stream's
    gradient d_h, of h's type) -> (d_x, d_y, d_w_pre, d_w_post, d_gate), None for parts that are not there.  d_x has h's
    type, d_y is bf16, the weights' gradients are fp32 [N]; d_gate is fp32 [N] for a gate [N] and bf16 [T, N] else.
    Equal calls give equal bits.  The call's partial sums (at most 52 MB) come from torch's allocator."""
    if stream is not None:
        return _on_stream(stream, residual_rms_norm_backward, d_z, h, w_pre, d_h, y, w_post, gate, residual_scale,
                          eps, weight_offset, d_x, d_y, d_w_pre, d_w_post, d_gate)
    T, N = _2d(h, "h")
    pz, ld_z = _rows(d_z, "d_z", _BF16, T, N)
    ph, ldh = _rows(h, "h", _FLOAT, T, N)
    pdh, ld_dh = (None, 0) if d_h is None else _rows(d_h, "d_h", (h.dtype,), T, N)
    if y is None and not (w_post is None and gate is None and d_y is None):
        raise ValueError("w_post, gate and d_y apply to y")
    if (w_post is None and d_w_post is not None) or (gate is None and d_gate is not None):
        raise ValueError("a gradient is asked for of a part that is not there")
    py, ldy = (None, 0) if y is None else _rows(y, "y", _BF16, T, N)
    pw = _whole(w_pre, "w_pre", _BF16, (N,))
    pwp = None if w_post is None else _whole(w_post, "w_post", _BF16, (N,))
    pg, ld_g = _gate(gate, T, N)
    d_x, pdx, ld_dx = _out_rows(d_x, "d_x", (h.dtype,), T, N, h)
    d_w_pre, pdw = _out(d_w_pre, "d_w_pre", _F32, (N,), h)
    pdy, ld_dy, pdwp, pdg, ld_dg = None, 0, None, None, 0
    if y is not None:
        d_y, pdy, ld_dy = _out_rows(d_y, "d_y", _BF16, T, N, h)
    if w_post is not None:
        d_w_post, pdwp = _out(d_w_post, "d_w_post", _F32, (N,), h)
    if gate is not None:
        if gate.dim() == 1:
            d_gate, pdg = _out(d_gate, "d_gate", _F32, (N,), h)
        else:
            d_gate, pdg, ld_dg = _out_rows(d_gate, "d_gate", _BF16, T, N, h)
    # partial sums from torch's allocator (the stream's, or a capture's own memory), not the library's workspace
    need = _lib.residual_rms_norm_backward_scratch_bytes(T, N)
    scratch = h.new_empty(need // 4, dtype=torch.float32) if need else None
    _launch("residual_rms_norm_backward_noalloc",
            (d_z, d_h, h, y, w_post, gate, w_pre), pz, ld_z, pdh, ld_dh, ph, ldh,
            h.dtype == torch.float32, py, ldy, pwp, pg, ld_g, pw, residual_scale, eps, weight_offset, T, N, pdx, ld_dx,
            pdy, ld_dy, pdw, pdwp, pdg, ld_dg, None if scratch is None else scratch.data_ptr(), need)
    return d_x, d_y, d_w_pre, d_w_post, d_gate


def silu_mul_quant_group_pack_checkpoint(x: torch.Tensor, masked_m: torch.Tensor, q: torch.Tensor | None = None,
                                         sf: torch.Tensor | None = None, cq: torch.Tensor | None = None,
                                         csf: torch.Tensor | None = None, stream=None):
    """silu_mul_quant_group_pack that also keeps gate and up in 8 bits for the backward pass.  x bf16
    [E, M_max, 2H], masked_m int32 [E] -> (q uint8 [E, M_max, H], sf int32 [E, ceil(H/512), M_max], cq uint8
    [E, M_max, 2H], csf int32 [E, 2 * ceil(H/512), M_max]); padded rows are not written."""
    if stream is not None:
        return _on_stream(stream, silu_mul_quant_group_pack_checkpoint, x, masked_m, q, sf, cq, csf)
    if x.dim() != 3 or x.shape[2] % 2:
        raise ValueError("x must be [E, M_max, 2H]")
    E, M_max, H2 = x.shape
    H, W = H2 // 2, _words(H2 // 2)
    px = _whole(x, "x", _BF16, x.shape)
    pm = _whole(masked_m, "masked_m", _I32, (E,))
    q, pq = _out(q, "q", _E4M3, (E, M_max, H), x)
    sf, psf = _out(sf, "sf", _U32, (E, W, M_max), x)
    cq, pc = _out(cq, "cq", _E4M3, (E, M_max, H2), x)
    csf, pcs = _out(csf, "csf", _U32, (E, 2 * W, M_max), x)
    _launch("silu_mul_quant_group_pack_checkpoint", (x, masked_m), px, pm, E, M_max, H, pq, psf,
            pc, pcs)
    return q, sf, cq, csf


def silu_mul_backward_from_checkpoint(d_y: torch.Tensor, masked_m: torch.Tensor, cq: torch.Tensor, csf: torch.Tensor,
                                      quantize: bool = False, d_x: torch.Tensor | None = None,
                                      q: torch.Tensor | None = None, sf: torch.Tensor | None = None, stream=None):
    """Gradient of silu(gate) * up from the 8-bit checkpoint: d_y bf16 [E, M_max, H] -> d_x bf16 [E, M_max, 2H], or
    with quantize (q uint8 [E, M_max, 2H], sf int32 [E, ceil(2H/512), M_max]) in the masked GEMM's layout; padded
    rows are not written."""
    if stream is not None:
        return _on_stream(stream, silu_mul_backward_from_checkpoint, d_y, masked_m, cq, csf, quantize, d_x, q, sf)
    if d_y.dim() != 3:
        raise ValueError("d_y must be [E, M_max, H]")
    E, M_max, H = d_y.shape
    W = _words(H)
    pd = _whole(d_y, "d_y", _BF16, d_y.shape)
    pm = _whole(masked_m, "masked_m", _I32, (E,))
    pc = _whole(cq, "cq", _E4M3, (E, M_max, 2 * H))
    pcs = _whole(csf, "csf", _U32, (E, 2 * W, M_max))
    px = pq = psf = None
    if quantize:
        if d_x is not None:
            raise ValueError("d_x is not written with quantize")
        q, pq = _out(q, "q", _E4M3, (E, M_max, 2 * H), d_y)
        sf, psf = _out(sf, "sf", _U32, (E, _words(2 * H), M_max), d_y)
    else:
        if q is not None or sf is not None:
            raise ValueError("q and sf are written with quantize only")
        d_x, px = _out(d_x, "d_x", _BF16, (E, M_max, 2 * H), d_y)
    _launch("silu_mul_backward_from_checkpoint", (d_y, masked_m, cq, csf), pd, pm, E, M_max, H, pc,
            pcs, px, pq, psf)
    return (q, sf) if quantize else d_x
