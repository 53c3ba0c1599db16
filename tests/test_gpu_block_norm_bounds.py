"""Block norms within the error of their own order of summation.

A thread squares and adds 8 elements (16 in rows of more than 8192) in fused
steps, four lane moves add 16 threads, all in fp32; whatever is added after that
is in fp64.  So a sum of squares, whose terms are all positive, is off by at
most n = 12 (20) times 2^-24 of itself; its mean's rounding and eps's addition
make n + 2, the root halves it, and the hardware's inverse root is off by one
step of the last place, 2^-23: (n + 2) / 2 + 2 = 9 (13).  Two products more:
|h - ref| <= 11 (15) 2^-24 |ref|, one more unit for the terms of second order.
After a block, gate, residual scale and sum each round once:
|out - ref| <= (11 (15) + 2 + 1) 2^-24 (|rs res| + |g b|).
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import test_gpu_block_norm as base

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
EPS = float(np.float32(1e-6))


def units(cols):
    return 12 if cols <= 8192 else 16


def rows_like(kind, cols, dtype, g):
    """Rows whose squares round alike, grow along the row, or are spread over many sizes."""
    n = torch.arange(cols, device=DEV)
    sign = torch.randint(0, 2, (6, cols), generator=g, device=DEV) * 2.0 - 1
    c = torch.rand((6, 1), generator=g, device=DEV) + 1.0
    x = {"alike": lambda: sign * c, "grows": lambda: sign * c * 2.0**(8.0 * n / cols),
         "spread": lambda: sign * torch.exp(2 * torch.randn((6, cols), generator=g, device=DEV)),
         "one": lambda: torch.where(n == cols // 2, 1000.0 * c, 1e-3 * sign)}[kind]()
    return x.to(dtype)


@pytest.mark.parametrize("kind", ["alike", "grows", "spread", "one"])
@pytest.mark.parametrize("cols", [1, 7, 63, 512, 513, 2049, 4096, 8192, 8193, 12000, 16384])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_within_the_order_of_summation(cols, kind, dtype):
    g = base.gen(cols)
    x = rows_like(kind, cols, dtype, g)
    w = 1 + 0.2 * torch.randn(cols, generator=g, device=DEV)
    want = ref.rms(ref.f64(x), ref.f64(w), EPS)
    h = m.moe_norm_pre(m.Norm(cols, pre_w=w), x, h_dtype=F32)
    base.close(h, want, np.abs(want), units(cols), F32)
    res = torch.randn((6, cols), generator=g, device=DEV)
    gate = 0.5 + 0.3 * torch.randn((6, 1), generator=g, device=DEV)
    out = m.moe_norm_post(m.Norm(cols, post_w=w, residual_scale=0.3), x, res, gate=gate)
    r, b = float(np.float32(0.3)) * ref.f64(res), want * ref.f64(gate)
    base.close(out, r + b, np.abs(r) + np.abs(b), units(cols) + 3, F32)


@pytest.mark.parametrize("cols", [2048, 8192, 16384])
def test_the_last_additions_lose_nothing(cols):
    """One element in each 128 (what 16 lanes add up), a whole number whose square fp32 holds:
    every sum in fp32 is exact, and so is the rest in fp64, so the order of the elements changes
    no bit.  Added in fp32 to the end, the orders' sums differ."""
    parts, rows = min(cols, 8192) // 128, 64
    rng = np.random.default_rng(cols)
    some = rng.choice(np.arange(2048, 4096), parts, replace=False)
    v = np.stack([rng.permutation(some) for _ in range(rows)])
    x = np.zeros((rows, cols), dtype=np.float32)
    x[:, np.arange(parts) * 128 + 17] = v
    s = (v * v).astype(np.float32)
    assert np.array_equal(s, (v.astype(np.int64) ** 2))
    while s.shape[1] > 1:
        s = s[:, ::2] + s[:, 1::2]
    assert len(np.unique(s)) > 1  # (the pairwise sums in fp32)
    x = torch.from_numpy(x).to(DEV)
    h = m.moe_norm_pre(m.Norm(cols), x).sort(dim=1).values
    assert (h == h[0]).all()
    y, res = x, torch.zeros_like(x)
    out, h2 = m.moe_norm_post(m.Norm(cols, post_norm=False), y, res, next_norm=m.Norm(cols))
    assert torch.equal(out, x) and torch.equal(h2.sort(dim=1).values, h)
