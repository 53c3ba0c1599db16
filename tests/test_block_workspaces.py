"""Workspace sizes of the block operators (CPU only): what the size functions
report for a number of rows serves every call of that many rows or fewer, so
one buffer for the largest chunk serves the smaller ones."""
import ctypes as C

import pytest
import torch

import mxfp4_routed_expert_e2m1_amd as m
from mxfp4_routed_expert_e2m1_amd import block as b

WORKSPACE = -4
A = 0x100000  # never dereferenced: without a GPU no call gets as far as a launch

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="accepted calls would be launched")


def rows_to(most):
    return sorted({r for r in range(1, min(most, 2200))} | set(range(2200, most, 977))
                  | {r for p in range(4, 25) for r in (2**p - 1, 2**p, 2**p + 1) if r <= most}
                  | {most})


@pytest.mark.parametrize("experts", [1, 8, 160, 256, 512])
def test_one_routing_workspace_serves_fewer_rows(experts):
    L, rule = m.lib(), b.moe_router_rule_t(experts, 1, 1, 1, 1, 1, 1, 1.0, None)
    rule = C.byref(rule)
    rows = rows_to(1 << 24)
    sizes = [L.moe_route_scored_workspace_bytes(rule, r) for r in rows]
    assert sizes == sorted(sizes)
    assert sizes[-1] <= 512 * 512 * 2
    for r, n in zip(rows, sizes):
        rc = L.moe_route_scored(rule, A, 0, experts, r, A, A, A, A, A, A, n, None)
        assert rc != WORKSPACE, f"{n} bytes are too few for {r} rows"
