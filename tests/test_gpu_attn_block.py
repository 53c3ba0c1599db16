"""The block with attention of examples/moe_block.py: the operators in the order in which a served block
uses them. Chunks of a prompt and single tokens give what the 64-bit form gives over the cache that
they wrote; other requests' tokens change nothing; a captured decode step replays as the texts grow."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import synth

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")
from examples.moe_block import AttentionBlock, Requests  # noqa: E402

SHAPE = synth.Layer(8, 2, 1024, 1024, True)
PAGE = 16


def make(n, most, window=0):
    return AttentionBlock(SHAPE, Requests(n, most, page=PAGE), seed=5, window=window)


def rows(n, step=0):
    return torch.from_numpy(synth.activations(5, step, n, SHAPE.d_model)).cuda()


def spy(block, x, step):
    """The block's mix with its queries and attention output kept."""
    kept, call = {}, m.moe_attn_cache

    def attn(desc, cache, q, *a, **kw):
        kept["q"], kept["o"] = q.clone(), call(desc, cache, q, *a, **kw)
        return kept["o"]
    m.moe_attn_cache = attn
    try:
        kept["u"] = block.mix(x, *step)
    finally:
        m.moe_attn_cache = call
    return kept


def check_attention(block, kept, new, window=0):
    """The attention's output against its formula over the values that the cache holds."""
    req, at = block.requests, 0
    for r, k in enumerate(new):
        n = req.lens[r]
        slots = torch.arange(n, dtype=torch.int32, device="cuda") + r * req.pages * req.page
        keys, values = m.moe_kv_read(block.cache, slots, dtype=torch.float32)
        q = ref.f64(kept["q"][at: at + k])
        scale = float(np.float32(block.dim ** -0.5))
        want, size, ds = ref.attention(q, ref.f64(keys), ref.f64(values), scale, window=window)
        err = ref.attention_error(size, ds, n, torch.bfloat16)
        ref.check(kept["o"][at: at + k], want, err, torch.bfloat16)
        at += k


@pytest.mark.parametrize("window", [0, 40])
def test_prompts_then_tokens(window):
    block = make(3, 200, window)
    for i, new in enumerate(([70, 33, 1], [1, 1, 1], [60, 0, 5], [1, 4, 1], [1, 1, 1])):
        step = block.requests.add(new)
        kept = spy(block, rows(sum(new), i), step)
        check_attention(block, kept, new, window)
        assert torch.isfinite(block.experts(rows(sum(new), i), kept["u"])).all()


def test_cached_keys_are_the_rotated_projection():
    """What the calls put in the cache: keys and values of the projection, keys rotated by their
    positions, in 4 bits."""
    block = make(1, 60)
    x = rows(50)
    step = block.requests.add([50])
    _, c, cs = m.moe_norm_pre(block.pre, x, h=False, quant="row")
    H, KV = block.heads, block.kv_heads
    qkv = m.moe_linear_q8(block.qkv, c, cs).view(50, H + 2 * KV, block.dim)
    k = m.moe_rope(block.rope, qkv[:, H: H + KV].contiguous(), step[0])
    kept = spy(block, x, step)
    keys, values = m.moe_kv_read(block.cache, step[1], dtype=torch.float32)
    assert np.array_equal(ref.f64(keys), ref.stored(ref.f64(k)))
    assert np.array_equal(ref.f64(values), ref.stored(ref.f64(qkv[:, H + KV:])))
    # the rotation turns a query and a key by their distance alone: the first row is not turned
    assert torch.equal(kept["q"][0], qkv[0, :H])


def test_a_request_does_not_depend_on_the_others():
    x = rows(40)
    alone, both = make(1, 100), make(2, 100)
    both.requests.add([0, 0])
    a = alone(x[:30], alone.requests.add([30]))
    b = both(torch.cat([x[:30], x[30:]]), both.requests.add([30, 10]))
    # (the same kernel for both: 30 and 40 rows of 2 key heads)
    assert torch.equal(a, b[:30])


def test_captured_decode_step_replays():
    """Texts grow by a token a step; the graph reads positions, slots and lengths where the eager
    step's are copied to."""
    block, twin = make(2, 400), make(2, 400)
    first = [37, 150]
    for b in (block, twin):
        b(rows(sum(first)), b.requests.add(first))
    x = rows(2, 1)
    held = [t.clone() for t in twin.requests.add([1, 1])[:3]]
    twin(x, (*held, None))
    twin.requests.lens = list(first)                       # (done again below)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = twin(x, (*held, None))
    for i in range(5):
        x.copy_(rows(2, 1 + i))
        step = block.requests.add([1, 1])
        for t, s in zip(held, step):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, block(x, step))
