"""The softmax weights of the attention over the 4-bit cache: what divides is the sum of what is added."""
import math

import numpy as np
import pytest
import torch

import attn_ref as ref
from test_gpu_attn import TYPES, call, i32, queries

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")

# (token, head) pairs of a sequence: single rows, 17 to 64, tiles of many rows; texts that are taken by
# one workgroup and ones that are cut
ROWS = [(1, 8), (5, 8), (40, 8), (1, 64)]
TEXTS = [130, 700, 5000]


def ones(n, dim, dtype, keys):
    paged = ref.Paged([n], 1, dim, 64, 31, dtype=dtype)
    paged.k[0][:] = keys(paged.k[0])
    paged.v[0].fill_(1.0)
    m.moe_kv_write(paged.cache, paged.k[0].cuda(), paged.v[0].cuda(), paged.slots[0].cuda())
    return paged


def check_ones(out, n, dtype):
    """Sums of n weights in two orders, each within n / 8 + 128 half steps of fp32 (attn_ref), and the
    division: in bf16 far less than half a step of the result, which is then 1 itself."""
    off = (2 * (n / 8 + 128) + 2) * 2.0**-24
    if dtype == torch.bfloat16:
        assert off < 2.0**-10 and (out == 1.0).all(), out.unique()
    else:
        assert (out.double() - 1).abs().max() <= off


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", TEXTS)
@pytest.mark.parametrize("new,heads", ROWS)
def test_weights_that_all_round_the_same_way(new, heads, n, dim, dtype):
    """Every 16th token weighs 1, all others 0.5 (1 + 2^-8 - 2^-12), which in 8 bits is 0.5: weights that
    are added in 8 bits and divided by the sum of unrounded ones would leave 1 - 2^-8."""
    def keys(k):
        k = torch.zeros_like(k)
        k[::16, :, 0] = 1.0
        return k
    paged = ones(n, dim, dtype, keys)
    q = torch.zeros((new, heads, dim), dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    scale = float(np.float32(-math.log(0.5 * (1 + 2.0**-8 - 2.0**-12))))
    check_ones(call(paged, q, [new], scale), n, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", TEXTS)
@pytest.mark.parametrize("new,heads", ROWS)
def test_equal_values_are_the_result(new, heads, n, dim, dtype):
    paged = ones(n, dim, dtype, lambda k: k)
    q = queries(new, heads, dim, dtype)
    check_ones(call(paged, q, [new], float(np.float32(dim ** -0.5))), n, dtype)
