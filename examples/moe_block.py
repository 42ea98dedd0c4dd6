"""One training step's pass through a mixture-of-experts block, forward and backward:

    norm after the block before, gate, scaled residual, norm before this one   (residual_rms_norm)
    router                                                                     (moe_route_topk)
    tokens to the experts' layout in e4m3                                      (fp8_quant_group_pack_to_experts)
    gate_up product, SiLU with an 8-bit checkpoint, down product               (masked GEMMs)
    experts' rows back to their tokens                                         (moe_combine)
    norm after, gate, residual, norm before the next block in e4m3             (residual_rms_norm)

and back: every activation's gradient, and those of the norms' weights, the gates and the
router.  (The experts' own weights have their gradients as products over the tokens, which
the library has no kernel for.)

    python examples/moe_block.py [--tokens 512] [--hidden 1024] [--half 512] [--experts 16] [--topk 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_fp8_token_amd as F  # noqa: E402

ROUTER = dict(scoring="sigmoid", renormalize=True, scale=1.5)


def quantized(w):
    """Expert weights bf16 [E, N, K] -> e4m3 [E, N, K] and 128x128 block scales."""
    E, N, K = w.shape
    q = torch.empty((E, N, K), dtype=torch.uint8, device=w.device)
    s = torch.empty((E, (N + 127) // 128, K // 128), dtype=torch.float32, device=w.device)
    for e in range(E):
        F.fp8_block_quant_128x128(w[e].contiguous(), q=q[e], sfb=s[e])
    return q, s


class MoeBlock:
    def __init__(self, hidden, half, experts, topk, groups=4, seed=0, device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)

        def r(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device=device) * std).to(torch.bfloat16)
        self.E, self.topk = experts, topk
        self.route = dict(groups=groups, topk_groups=groups // 2, group_top=2, **ROUTER)
        self.router = r(experts, hidden, std=hidden ** -0.5)
        self.bias = torch.zeros(experts, device=device)  # moved by whoever balances the load
        self.w_gate_up = r(experts, 2 * half, hidden, std=hidden ** -0.5)
        self.w_down = r(experts, hidden, half, std=half ** -0.5)
        # each product's weights, and transposed for the gradient of its input, once
        self.gate_up, self.down = quantized(self.w_gate_up), quantized(self.w_down)
        self.gate_up_t = quantized(self.w_gate_up.transpose(1, 2))
        self.down_t = quantized(self.w_down.transpose(1, 2))
        self.norms = {n: r(hidden, std=0.1) + 1 for n in ("post0", "pre0", "post1", "pre1")}
        self.gates = {n: r(hidden, std=0.3) + 1 for n in ("gate0", "gate1")}

    def forward(self, x, y, capacity):
        """Residual stream x and the output y of the block before, bf16 [T, hidden] -> the new stream and the
        next block's input in e4m3 (codes, scale words), and what the backward pass needs."""
        n, g = self.norms, self.gates
        h, z, _, _ = F.residual_rms_norm(x, n["pre0"], y=y, w_post=n["post0"], gate=g["gate0"])
        logits = torch.mm(z, self.router.t())
        ids, w = F.moe_route_topk(logits, self.topk, bias=self.bias, **self.route)
        q, sf, rows, slots = F.fp8_quant_group_pack_to_experts(z, ids, self.E, capacity)
        gate_up = F.fp8_block_gemm_grouped_masked(q, sf, *self.gate_up, rows)
        q, sf, cq, csf = F.silu_mul_quant_group_pack_checkpoint(gate_up, rows)
        experts = F.fp8_block_gemm_grouped_masked(q, sf, *self.down, rows)
        out = F.moe_combine(experts, ids, slots, w)
        h1, _, q, sf = F.residual_rms_norm(h, n["pre1"], y=out, w_post=n["post1"], gate=g["gate1"], out="fp8")
        kept = dict(y=y, h=h, logits=logits, ids=ids, w=w, rows=rows, slots=slots, cq=cq, csf=csf, experts=experts,
                    out=out, h1=h1)
        return h1, q, sf, kept

    def backward(self, d_h1, d_z1, s):
        """Gradients of the new stream and of the next block's input -> those of x and y, and of the weights
        named in `norms`, `gates` and `router`."""
        n, g, d = self.norms, self.gates, {}
        d_h, d_out, d["pre1"], d["post1"], d["gate1"] = F.residual_rms_norm_backward(
            d_z1, s["h1"], n["pre1"], d_h=d_h1, y=s["out"], w_post=n["post1"], gate=g["gate1"])
        q, sf, d_w = F.moe_combine_backward(d_out, s["experts"], s["ids"], s["slots"], s["w"], quantize=True)
        d_act = F.fp8_block_gemm_grouped_masked(q, sf, *self.down_t, s["rows"])
        q, sf = F.silu_mul_backward_from_checkpoint(d_act, s["rows"], s["cq"], s["csf"], quantize=True)
        d_tokens = F.fp8_block_gemm_grouped_masked(q, sf, *self.gate_up_t, s["rows"])
        d_logits = F.moe_route_topk_backward(s["logits"], s["ids"], d_w, **ROUTER)
        # the dispatch's gradient: the experts' rows summed per token, on top of the router's part
        d_z = F.moe_combine(d_tokens, s["ids"], s["slots"], base=torch.mm(d_logits, self.router))
        # (the norm's output is not kept: it is one pass over the stream that is)
        _, z, _, _ = F.residual_rms_norm(s["h"], n["pre0"])
        d["router"] = torch.mm(d_logits.t(), z)
        d["x"], d["y"], d["pre0"], d["post0"], d["gate0"] = F.residual_rms_norm_backward(
            d_z, s["h"], n["pre0"], d_h=d_h, y=s["y"], w_post=n["post0"], gate=g["gate0"])
        return d


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 512), ("hidden", 1024), ("half", 512), ("experts", 16), ("topk", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    block = MoeBlock(a.hidden, a.half, a.experts, a.topk)
    x, y, d_h, d_z = (torch.randn(a.tokens, a.hidden, device="cuda:0").to(torch.bfloat16) for _ in range(4))
    capacity = min(a.tokens, (2 * a.tokens * a.topk // a.experts + 15) // 16 * 16)
    h, q, sf, kept = block.forward(x, y, capacity)
    grads = block.backward(d_h, d_z, kept)
    dropped = int((kept["slots"] < 0).sum())
    print("tokens %d, pairs %d (%d over the capacity of %d)" % (a.tokens, a.tokens * a.topk, dropped, capacity))
    print("stream rms %.3f" % h.float().square().mean().sqrt().item())
    for name, t in grads.items():
        print("d_%-6s %-14s rms %.3g" % (name, list(t.shape), t.float().square().mean().sqrt().item()))


if __name__ == "__main__":
    main()
