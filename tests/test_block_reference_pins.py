"""The references that the GPU tests of the operators around the experts' products use, pinned
on the CPU: against torch where it has the operation, and against planted mistakes."""
import numpy as np
import pytest
import torch

import block_reference as R


def rng(*seed):
    return np.random.default_rng([30, *seed])


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_against_topk(scoring, renormalize):
    l = rng(1).normal(size=(20, 48))
    b = rng(2).normal(size=48)
    t = torch.from_numpy(l)
    s = torch.sigmoid(t) if scoring == "sigmoid" else torch.softmax(t, 1)
    for bias in (None, b):
        ids, w, gap = R.route(l, 5, bias=bias, scoring=scoring, renormalize=renormalize, scale=3.0)
        want = torch.topk(s if bias is None else s + torch.from_numpy(bias), 5, dim=1).indices
        c = s.gather(1, want)
        c = 3.0 * (c / c.sum(1, keepdim=True) if renormalize else c)
        assert gap > 0 and np.array_equal(ids, want.numpy())
        assert np.allclose(w, c.numpy(), rtol=1e-12)
        assert np.allclose(R.route_weights(l, ids, scoring, renormalize, 3.0), w, rtol=1e-12)


def test_route_groups_by_hand():
    # groups {3, 1}, {2, 2.5}, {0, 4}: best ranks 3, 2.5, 4; sums of two sigmoids 1.68, 1.80, 1.48
    l = np.array([[3.0, 1.0, 2.0, 2.5, 0.0, 4.0]])
    assert R.route(l, 2, groups=3, topk_groups=1, group_top=1)[0].tolist() == [[5, 4]]
    assert R.route(l, 2, groups=3, topk_groups=1, group_top=2, scoring="sigmoid")[0].tolist() == [[3, 2]]
    l[0, 5] = -np.inf  # the third group is left with one expert
    assert R.route(l, 3, groups=3, topk_groups=2, group_top=1)[0].tolist() == [[0, 3, 2]]
    assert R.route(np.full((1, 4), np.nan), 2)[0].tolist() == [[-1, -1]]


def test_combine_against_einsum():
    g = rng(3)
    y, w = g.normal(size=(3, 4, 8)), g.random((5, 2))
    ids, slots = g.integers(0, 3, (5, 2)), g.integers(0, 4, (5, 2))
    out, _ = R.combine(y, ids, slots, w, None)
    assert np.allclose(out, np.einsum("tj,tjn->tn", w, y[ids, slots]))
    slots[2, 1] = -1
    assert np.allclose(R.combine(y, ids, slots, w, None)[0][2], w[2, 0] * y[ids[2, 0], slots[2, 0]])


def test_norm_against_torch():
    g = rng(4)
    x, y, w, v, gate = (g.normal(size=s) for s in ((3, 32), (3, 32), 32, 32, 32))
    h, z = R.norm(x, w, y, v, gate, 0.5, 1e-3, 1.0)
    t = torch.from_numpy
    want = 0.5 * t(x) + t(gate) * torch.nn.functional.rms_norm(t(y), (32,), t(v) + 1, 1e-3)
    assert np.allclose(h, want) and np.allclose(z, torch.nn.functional.rms_norm(want, (32,), t(w) + 1, 1e-3))


def quantized(v):
    """Codes and words of v [rows, K] by torch's own cast."""
    rows, K = v.shape
    gr = v.reshape(rows, -1, 128)
    need = np.maximum(np.abs(gr).max(-1), 1e-10) / 448
    e = np.ceil(np.log2(need)).astype(np.int64)
    codes = torch.from_numpy(gr / 2.0 ** e[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    b = np.zeros((rows, -(-e.shape[1] // 4) * 4), np.uint32)
    b[:, :e.shape[1]] = e + 127
    b = b.reshape(rows, -1, 4)
    words = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | b[..., 3] << 24
    return codes.reshape(rows, K).numpy().copy(), np.ascontiguousarray(words.T.astype(np.uint32))


def test_decode_is_torchs():
    c = np.arange(256, dtype=np.uint8)
    c = c[(c & 0x7F) != 0x7F]
    assert np.array_equal(R.e4m3_decode(c), torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy())


def test_check_quantized_sees_planted_mistakes():
    v = rng(5).normal(size=(4, 640)).astype(np.float32).astype(np.float64)
    codes, words = quantized(v)
    R.check_quantized(v, codes, words, 0.0)
    for plant in range(5):
        c, w = codes.copy(), words.copy()
        if plant == 0:
            c[2, 77] ^= 0x80            # a sign
        elif plant == 1:
            c[1, 300] += 1              # a neighbour
        elif plant == 2:
            w[0, 3] += 1                # a scale of twice the size
        elif plant == 3:
            w[0, 3] -= 1 << 8           # and of half
        else:
            w[1, 0] |= 1 << 16          # a byte past the row's groups
        with pytest.raises(AssertionError):
            R.check_quantized(v, c, w, 1e-9)
