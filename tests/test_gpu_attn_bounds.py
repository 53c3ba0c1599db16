"""What calls of the attention over the 4-bit cache may touch where offsets and lengths are wrong: `out`
and the workspace lie in larger tensors of a known pattern."""
import pytest
import torch

import attn_ref as ref
from test_gpu_attn import TYPES, i32, queries

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")

GUARD = 4096


class Guarded:
    """A tensor in the middle of a larger one, and whether the rest is as it was."""

    def __init__(self, shape, dtype, fill):
        n = 1
        for s in shape:
            n *= s
        self.whole = torch.full((n + 2 * GUARD,), fill, dtype=dtype, device="cuda")
        self.t = self.whole[GUARD: GUARD + n].view(shape)
        self.fill = fill

    def intact(self):
        ends = torch.cat([self.whole[:GUARD], self.whole[-GUARD:]])
        return bool((ends == self.fill).all())


def least_workspace(go):
    """The bytes that a call does not refuse."""
    low, high = -1, 1 << 30
    while high - low > 1:
        n = (low + high) // 2
        try:
            go(n)
            high = n
        except m.MoeError:
            low = n
    return high


def rows_of(off, rows):
    """The rows that some sequence has after its offsets are kept in 0..rows."""
    have = set()
    off = [min(max(o, 0), rows) for o in off]
    for a, b in zip(off, off[1:]):
        have |= set(range(a, b))
    return have


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,rows,heads", [([64, 50, 3], 6, 2),          # one workgroup a text
                                             ([5000, 4000, 700], 6, 2),    # cut, few rows
                                             ([256, 200, 90], 160, 2),     # many rows
                                             ([5000, 4000, 700], 300, 8)]) # many rows, cut
def test_offsets_that_go_back_or_lie_outside(lens, rows, heads, dtype):
    paged = ref.Paged(lens, 1, 64, 64, 40, dtype=dtype)
    # (lengths past the table's end: every entry is a page)
    paged.table.clamp_(0, paged.cache.n_pages - 1)
    q = queries(rows, heads, 64, dtype)
    attn = m.Attention(heads, 0.125)
    table = paged.table.cuda()
    big = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    offsets = i32([0, rows, rows, rows])

    def plain(n):
        m.moe_attn_cache(attn, paged.cache, q, table, i32(lens), q_offsets=offsets,
                         ws=big[:min(n, 1 << 26)])
    need = least_workspace(plain)
    assert (need > 0) == (lens[0] == 5000)
    half = rows // 2
    for off in ([0, rows, half, rows], [rows, 0, rows, 0], [half, half, 1, 0], [-9, -3, 0, 0],
                [0, rows, 0, rows], [-5, 2, 10**9, 2**31 - 1], [0, half, rows, 10**6], [0, 2, 2, 4]):
        for kv in (lens, [10**9, -3, 2**31 - 1], [0, 0, 0]):
            out = Guarded((rows, heads, 64), dtype, 3.0)
            ws = Guarded((need,), torch.uint8, 0x5A)
            m.moe_attn_cache(attn, paged.cache, q, table, i32(kv), q_offsets=i32(off), out=out.t, ws=ws.t)
            torch.cuda.synchronize()
            assert out.intact() and ws.intact(), (off, kv)
            others = sorted(set(range(rows)) - rows_of(off, rows))
            assert (out.t[others] == 3.0).all(), (off, kv)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,new,heads", [([64, 50], [1, 3], 2), ([5000, 4000], [1, 3], 2),
                                            ([5000, 4000], [5, 5], 8), ([256, 200], [90, 70], 2),
                                            ([5000, 4000], [60, 240], 8)])
def test_the_least_workspace_and_nothing_else(lens, new, heads, dim, dtype):
    """A call with no byte more than it asks for, between guards, is right."""
    paged = ref.Paged(lens, 1, dim, 64, 41, dtype=dtype)
    rows = sum(new)
    q = queries(rows + 3, heads, dim, dtype)
    attn = m.Attention(heads, 0.125)
    table, off = paged.table.cuda(), i32([0, new[0], rows])
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def go(n, out=None, ws=None):
        return m.moe_attn_cache(attn, paged.cache, q, table, i32(lens), q_offsets=off, out=out,
                                ws=big[:min(n, 1 << 28)] if ws is None else ws)
    need = least_workspace(go)
    assert need <= m.moe_attn_cache_workspace_bytes(attn, paged.cache, rows + 3, 2)
    out, ws = Guarded((rows + 3, heads, dim), dtype, 3.0), Guarded((need,), torch.uint8, 0x5A)
    go(need, out.t, ws.t)
    assert out.intact() and ws.intact() and (out.t[rows:] == 3.0).all()
    assert torch.equal(out.t[:rows], go(1 << 28)[:rows])
    ref.check_batch(out.t[:rows], paged, q, new, dtype, 0.125)
