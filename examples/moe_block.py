#!/usr/bin/env python3
"""One block with routed experts, from residual stream to residual stream.

    h, codes      = norm before the dense projection, quantised per row
    u             = int8 projection of the codes
    x1, h, codes  = x + gate * norm(u), and in the same pass the norm before the
                    experts, quantised per 32 elements
    logits, route = router projection, scored routing with a balance bias
    y             = routed experts (and the shared one)
    x2            = x1 + gate * norm(y)

The dense projection stands for whatever mixes a block's tokens.  Run on a GPU:

    python examples/moe_block.py --rows 1        # a decoded token
    python examples/moe_block.py --rows 512      # a prefill chunk
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import mxfp4_routed_expert_e2m1_amd as m  # noqa: E402
import synth  # noqa: E402


class Block:
    """Weights and descriptors of one block, made from a seed."""

    def __init__(self, shape, seed=0, device="cuda"):
        D, E = shape.d_model, shape.n_experts
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        weight = lambda: 1 + 0.1 * rand(D)  # noqa: E731
        self.pre = m.Norm(D, pre_w=weight())
        self.post = m.Norm(D, post_w=weight(), residual_scale=1.0)
        self.pre_experts = m.Norm(D, pre_w=weight())
        self.post_experts = m.Norm(D, post_w=weight(), residual_scale=1.0)
        self.gate, self.gate_experts = 0.5 + 0.1 * rand(D), 0.5 + 0.1 * rand(D)
        self.proj = m.Linear(*m.moe_quant_row_q8(rand(D, D) * D ** -0.5))
        self.router = (rand(E, D) * D ** -0.5).to(torch.bfloat16)
        groups = 8 if E % 8 == 0 and E >= 64 else 1
        self.rule = m.RouterRule(E, shape.top_k, score="sigmoid", bias=0.05 * rand(E),
                                 n_groups=groups, top_groups=max(1, groups // 2),
                                 group_score="top2", renorm=True, scale=2.5)
        experts = lambda e: synth.expert_weights(seed, 0, e, D, shape.d_ff, device=device)  # noqa: E731
        self.layer = m.pack_layer(D, shape.d_ff, E, shape.top_k, experts,
                                  has_shared=shape.has_shared, device=device)

    def __call__(self, x):
        """The block's output for the rows x [rows][d_model] (f32) of the residual stream."""
        _, q, qs = m.moe_norm_pre(self.pre, x, h=False, quant="row")
        u = m.moe_linear_q8(self.proj, q, qs)
        x1, h, q, qs = m.moe_norm_post(self.post, u, x, gate=self.gate,
                                       next_norm=self.pre_experts, quant="block")
        logits = m.moe_router_logits(h, self.router)
        ids, w, counts, offsets, srt = m.moe_route_scored(self.rule, logits)
        ffn = m.moe_ffn_decode if len(x) <= m.MOE_MAX_DECODE_ROWS else m.moe_ffn_prefill
        y = ffn(self.layer, q, qs, ids, w, offsets, srt)
        return m.moe_norm_post(self.post_experts, y, x1, gate=self.gate_experts)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=1)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tiny", action="store_true", help="8 experts of 256 x 512")
    a = ap.parse_args()
    shape = synth.TINY["layer"] if a.tiny else synth.DSV4_LAYER
    block = Block(shape)
    x = torch.from_numpy(synth.activations(0, 0, a.rows, shape.d_model)).cuda()
    y = block(x)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        y = block(x)
    torch.cuda.synchronize()
    us = (time.perf_counter() - t) / a.steps * 1e6
    print(f"{a.rows} rows of {shape.d_model}, {shape.n_experts} experts: {us:.1f} us a block, "
          f"rms in {float(x.square().mean().sqrt()):.3f} out {float(y.square().mean().sqrt()):.3f}")


if __name__ == "__main__":
    main()
