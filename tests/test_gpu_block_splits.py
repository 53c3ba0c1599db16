"""int8 linear layer where K is split over workgroups: rows that end inside a
step of K, splits of unequal length, odd channels, a bias in the launch that
joins the sums.  Bit for bit, as the sums are exact and every later step is one
rounded fp32 operation."""
import numpy as np
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
WORKSPACE = -4


def layer(rows, n, k, bias, seed=0):
    """Random codes, with random bytes past each row's end."""
    rng = np.random.default_rng([rows, n, k, seed])
    ld = (k + 15) // 16 * 16
    q, w = (rng.integers(-128, 128, (c, ld), dtype=np.int8) for c in (rows, n))
    qs, ws = (rng.uniform(0.5, 2.0, c).astype(np.float32) * 2.0**-10 for c in (rows, n))
    b = rng.standard_normal(n).astype(np.float32) if bias else None
    dev = lambda v: None if v is None else torch.from_numpy(v).to(DEV)  # noqa: E731
    lay = m.Linear(dev(w)[:, :k], dev(ws), dev(b))
    return lay, dev(q)[:, :k], dev(qs), lambda dt: ref.linear(q[:, :k], w[:, :k], qs, ws, b, dt)


def bytes_of(splits, rows, n):
    return splits * rows * ((n + 3) // 4 * 4) * 4


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,n,k,splits", [
    (48, 1000, 14000, 8), (100, 1001, 11058, 8), (64, 513, 8200, 8), (200, 300, 5000, 8),
    (130, 70, 4099, 8), (300, 1000, 14001, 4), (17, 4001, 6001, 4), (364, 991, 8397, 2),
    (254, 1667, 11192, 2), (117, 2479, 8923, 2)])
def test_splits_of_ragged_rows(rows, n, k, splits, dtype):
    need = bytes_of(splits, rows, n)
    for bias in (True, False):
        lay, q, qs, want = layer(rows, n, k, bias)
        assert m.moe_linear_q8_workspace_bytes(lay, rows) >= need
        with pytest.raises(m.MoeError) as e:  # (the call does split K so many ways)
            m.moe_linear_q8(lay, q, qs, dtype=dtype,
                            ws=torch.empty(need - 16, dtype=torch.uint8, device=DEV))
        assert e.value.status == WORKSPACE
        whole = torch.full((rows + 1, n + 3), 9.0, dtype=dtype, device=DEV)
        ws = torch.full((need + 256,), 77, dtype=torch.uint8, device=DEV)
        y = m.moe_linear_q8(lay, q, qs, y=whole[:rows, :n], ws=ws[:need])
        assert torch.equal(y.cpu(), want(dtype))
        assert (whole[rows] == 9).all() and (whole[:, n:] == 9).all() and (ws[need:] == 77).all()


def test_one_workspace_for_all_chunks():
    """Sized for the largest chunk, it serves smaller ones, split or not, in any order."""
    n, k, most = 1000, 14001, 700
    lay, q, qs, want = layer(most, n, k, True)
    want = want(F32)
    ws = torch.empty(m.moe_linear_q8_workspace_bytes(lay, most), dtype=torch.uint8, device=DEV)
    for rows in (700, 1, 17, 48, 64, 65, 128, 300, 511, 512, 513, 16, 699):
        y = m.moe_linear_q8(lay, q[:rows], qs[:rows], dtype=F32, ws=ws)
        assert torch.equal(y.cpu(), want[:rows]), f"{rows} rows"
    rule = m.RouterRule(256, 8)
    z = torch.randn((1100, 256), device=DEV)
    ws = torch.empty(m.moe_route_scored_workspace_bytes(rule, 1100), dtype=torch.uint8, device=DEV)
    ids, w, *_ = m.moe_route_scored(rule, z, ws=ws)
    for rows in (1024, 1025, 17, 33, 500, 1099):
        got = m.moe_route_scored(rule, z[:rows], ws=ws)
        assert torch.equal(got[0], ids[:rows]) and torch.equal(got[1], w[:rows])
