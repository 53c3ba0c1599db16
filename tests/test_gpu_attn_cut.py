"""Attention over the 4-bit cache where its tokens are cut into pieces: texts of hundreds of millions of
tokens."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from test_gpu_attn import i32, queries

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")


def test_a_text_of_300_million_tokens():
    """More work than 2^25 steps of 64 tokens: 128 heads on one, 8 tiles of 16 in f32, whose table
    repeats 4 pages, so that the result is that of those pages' tokens, each of the same weight.  Errors
    are those of a piece, of less than 8 n / 700 tokens (768 of them, over 8 tiles)."""
    heads, dim, page, dtype = 128, 64, 256, torch.float32
    paged = ref.Paged([4 * page], 1, dim, page, 30, spare=0)
    times = 293000
    n = times * 4 * page
    table = paged.table.cuda().repeat(1, times)
    q = queries(1, heads, dim, dtype)
    out = torch.full_like(q, 7.0)
    scale = float(np.float32(dim ** -0.5))
    m.moe_attn_cache(m.Attention(heads, scale), paged.cache, q, table, i32([n]), out=out)
    want, size, ds = ref.attention(ref.f64(q), *paged.values(0), scale)
    ref.check(out, want, ref.attention_error(size, ds, 8 * n / 700, dtype), dtype)
