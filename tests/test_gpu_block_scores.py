"""Scored routing: the scores' bits, and expert groups so large that 32 lanes
share one."""
import numpy as np
import pytest
import torch

import oracle
import test_gpu_block_route as base

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")
F32 = np.float32
ONE = F32(1)


def swept(n, rng):
    """Logits over and past the exponential's range, whole numbers and halves among them."""
    z = np.concatenate([rng.uniform(-110, 110, n // 2), rng.uniform(-12, 12, n // 4),
                        rng.standard_normal(n // 4 - 512) * 1e-3, np.arange(-128, 128) / 1.0,
                        np.arange(-128, 128) / 2.0]).astype(F32)
    return rng.permutation(z)


@pytest.mark.parametrize("rows", [16, 640, 1 << 16])
def test_sigmoid_scores_have_the_fixed_exponentials_bits(rows):
    """The weights are 1 / (1 + exp(-l)) in fp32 with the exponential that the experts'
    activation takes (the oracle repeats it operation for operation)."""
    z = swept(max(16 * rows, 4096), np.random.default_rng(rows))[:16 * rows].reshape(rows, 16)
    ids, w, *_ = base.run(z, m.RouterRule(16, 16, renorm=False))
    with np.errstate(over="ignore"):
        s = ONE / (ONE + oracle.exp_rows(-z).reshape(z.shape))
    assert np.array_equal(np.sort(ids, axis=1), np.tile(np.arange(16), (rows, 1)))
    assert np.array_equal(w.view(np.int32), np.take_along_axis(s, ids, 1).view(np.int32))


@pytest.mark.parametrize("rows", [16, 640, 1 << 16])
def test_softmax_scores_have_the_fixed_exponentials_bits(rows):
    z = swept(max(2 * rows, 4096), np.random.default_rng(rows + 1))[:2 * rows].reshape(rows, 2)
    ids, w, *_ = base.run(z, m.RouterRule(2, 2, score="softmax", renorm=False))
    e = oracle.exp_rows(z - z.max(axis=1, keepdims=True)).reshape(z.shape)
    s = e / (e[:, :1] + e[:, 1:])
    assert np.array_equal(w.view(np.int32), np.take_along_axis(s, ids, 1).view(np.int32))


@pytest.mark.parametrize("rows", [1, 9, 100, 333])
@pytest.mark.parametrize("experts", [256, 510, 130, 64, 34])
@pytest.mark.parametrize("group_score", ["top2", "max"])
def test_two_large_groups(rows, experts, group_score):
    """Two groups of up to 256 experts, the better one by its two largest keys wherever in the
    group they are."""
    rng = np.random.default_rng([rows, experts])
    kw = dict(top_k=6, score="sigmoid", n_groups=2, top_groups=1, group_score=group_score)
    z = base.logits(rng, rows, experts, kw, None, torch.float32)
    base.check(z, kw)
    # the two groups' largest keys alike, and the second largest of one in each of its places
    half = experts // 2
    z = np.full((half, experts), -3.0, dtype=F32)
    at = np.arange(half)
    z[:, 0], z[:, half + 5] = 2.0, 2.0
    z[at, half + (5 + at) % half] = np.where(at == 0, 2.0, 1.0)
    ids = base.check(z, dict(kw, top_k=2, group_score=group_score))
    if group_score == "top2":
        assert list(ids[1:, 1]) == list(half + (5 + at[1:]) % half)
