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


SHAPES = [(4096, 4096), (4096, 14336), (14336, 4096), (2048, 4096), (70, 4096), (130, 65536),
          (1, 8192), (1000, 14000), (1001, 11058), (513, 8200), (300, 5000), (64, 1025),
          (33, 65536), (12288, 4096), (20000, 65536), (32768, 2000), (256, 1000), (8, 64)]


@pytest.mark.parametrize("n_out,d_in", SHAPES)
def test_one_linear_workspace_serves_fewer_rows(n_out, d_in):
    L = m.lib()
    ld = (d_in + 15) // 16 * 16
    lay = C.byref(b.moe_linear_t(n_out, d_in, A, ld, A, None))
    rows = rows_to(40000)
    sizes = [L.moe_linear_q8_workspace_bytes(lay, r) for r in rows]
    assert sizes == sorted(sizes)
    call = lambda r, n: L.moe_linear_q8(lay, A, ld, A, r, A, 0, n_out, A, n, None)  # noqa: E731
    for r, n in zip(rows, sizes):
        assert call(r, n) != WORKSPACE, f"{n} bytes are too few for {r} rows"
    # and it is no more than a call of that size: within 64 rows of one that needs it all
    need = max((n for r in rows for n in [need_of(call, r)]), default=0)
    assert need <= sizes[-1] <= need * (1 + 64 / 17)


def need_of(call, rows):
    """The fewest bytes that a call takes (a multiple of 16, by bisection)."""
    lo, hi = -1, 1 << 28
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if call(rows, mid) == WORKSPACE else (lo, mid)
    return hi
