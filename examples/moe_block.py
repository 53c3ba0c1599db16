#!/usr/bin/env python3
"""One block with routed experts, from residual stream to residual stream.

    h, codes      = norm before the dense projection, quantised per row
    u             = int8 projection of the codes
    x1, h, codes  = x + gate * norm(u), and in the same pass the norm before the
                    experts, quantised per 32 elements
    logits, route = router projection, scored routing with a balance bias
    y             = routed experts (and the shared one)
    x2            = x1 + gate * norm(y)

The dense projection stands for whatever mixes a block's tokens.  With attention (AttentionBlock),
it is

    q, k, v       = int8 projection of the codes, rotary positions on q and k
    cache         = k and v into the request's pages, 4 bits a channel
    u             = int8 projection of the attention over the cached tokens

Run on a GPU:

    python examples/moe_block.py --rows 1        # a decoded token
    python examples/moe_block.py --rows 512      # a prefill chunk
    python examples/moe_block.py --rows 16 --context 8192    # 16 requests, a token each
    python examples/moe_block.py --rows 512 --context 8192   # a chunk of one request
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
        return self.experts(x, m.moe_linear_q8(self.proj, q, qs))

    def experts(self, x, u):
        """The rest of the block, from what mixes its tokens."""
        x1, h, q, qs = m.moe_norm_post(self.post, u, x, gate=self.gate,
                                       next_norm=self.pre_experts, quant="block")
        logits = m.moe_router_logits(h, self.router)
        ids, w, counts, offsets, srt = m.moe_route_scored(self.rule, logits)
        ffn = m.moe_ffn_decode if len(x) <= m.MOE_MAX_DECODE_ROWS else m.moe_ffn_prefill
        y = ffn(self.layer, q, qs, ids, w, offsets, srt)
        return m.moe_norm_post(self.post_experts, y, x1, gate=self.gate_experts)


class Requests:
    """Pages and lengths of requests of up to `most` tokens each, and what a step that adds tokens to
    them hands to the calls."""

    def __init__(self, n, most, page=64, device="cuda"):
        self.n, self.page, self.device = n, page, device
        self.pages = -(-most // page)
        self.table = torch.arange(n * self.pages, dtype=torch.int32, device=device).view(n, -1)
        self.lens = [0] * n

    def add(self, new):
        """(positions, slots, lens, q_offsets) for new[r] more tokens of request r."""
        at = [n + i for n, k in zip(self.lens, new) for i in range(k)]
        request = [r for r, k in enumerate(new) for _ in range(k)]
        self.lens = [n + k for n, k in zip(self.lens, new)]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=self.device)  # noqa: E731
        slots = [r * self.pages * self.page + i for r, i in zip(request, at)]
        ends = [sum(new[:r]) for r in range(self.n + 1)]
        return i32(at), i32(slots), i32(self.lens), None if new == [1] * self.n else i32(ends)


class AttentionBlock(Block):
    """A block whose tokens are mixed by attention over a cache in 4 bits: 4 query heads to a key
    head, rotary positions, a window where one is given."""

    def __init__(self, shape, requests, seed=0, window=0, device="cuda"):
        super().__init__(shape, seed, device)
        D = shape.d_model
        g = torch.Generator(device=device)
        g.manual_seed(seed + 1)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.requests, self.dim = requests, 128 if D >= 1024 else 64
        self.heads = D // self.dim
        self.kv_heads = max(1, self.heads // 4)
        wide = (self.heads + 2 * self.kv_heads) * self.dim
        self.qkv = m.Linear(*m.moe_quant_row_q8(rand(wide, D) * D ** -0.5))
        self.out = m.Linear(*m.moe_quant_row_q8(rand(D, D) * D ** -0.5))
        self.rope = m.Rope([10000.0 ** (-2 * i / self.dim) for i in range(self.dim // 2)],
                           device=device)
        self.attn = m.Attention(self.heads, scale=self.dim ** -0.5, window=window)
        self.cache = m.KVCache(requests.n * requests.pages, requests.page, self.kv_heads, self.dim,
                               device=device)

    def mix(self, x, positions, slots, lens, q_offsets):
        _, c, cs = m.moe_norm_pre(self.pre, x, h=False, quant="row")
        H, KV = self.heads, self.kv_heads
        qkv = m.moe_linear_q8(self.qkv, c, cs).view(len(x), H + 2 * KV, self.dim)
        rotated = qkv[:, : H + KV]
        m.moe_rope(self.rope, rotated, positions, out=rotated)
        m.moe_kv_write(self.cache, qkv[:, H: H + KV], qkv[:, H + KV:], slots)
        o = m.moe_attn_cache(self.attn, self.cache, qkv[:, :H], self.requests.table, lens, q_offsets)
        return m.moe_linear_q8(self.out, *m.moe_quant_row_q8(o.view(len(x), -1)))

    def __call__(self, x, step):
        """The block's output for the rows x of a step (Requests.add)."""
        return self.experts(x, self.mix(x, *step))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=1)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--context", type=int, default=0,
                    help="tokens in the cache of each request (0: a block without attention); up to 16 "
                         "rows are a request each, more are a chunk of one")
    ap.add_argument("--tiny", action="store_true", help="8 experts of 256 x 512")
    a = ap.parse_args()
    shape = synth.TINY["layer"] if a.tiny else synth.DSV4_LAYER
    x = torch.from_numpy(synth.activations(0, 0, a.rows, shape.d_model)).cuda()
    if a.context:
        single = a.rows <= m.MOE_MAX_DECODE_ROWS
        requests = Requests(a.rows if single else 1, a.context + a.rows)
        whole = AttentionBlock(shape, requests)
        requests.add([a.context] * requests.n)      # (their tokens: zeros, which a new cache holds)
        step = requests.add([1] * a.rows if single else [a.rows])
        block = lambda rows: whole(rows, step)  # noqa: E731
    else:
        block = Block(shape)
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
