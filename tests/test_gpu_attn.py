"""Attention over the 4-bit cache against its 64-bit form: types, head layouts, lengths from none to
long ones, pages that end inside a tile, windows, prefixes, caps and biases, what lies in masked
places, cut and uncut calls, strides, streams, replays."""
import numpy as np
import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")

TYPES = [torch.float32, torch.bfloat16]


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32, device="cuda")


def queries(rows, heads, dim, dtype, seed=1, grow=1.0):
    g = torch.Generator().manual_seed(seed)
    return (grow * torch.randn(rows, heads, dim, generator=g)).to(dtype).cuda()


def offsets(new):
    return i32(np.concatenate([[0], np.cumsum(new)]))


def call(paged, q, new, scale, softcap=0.0, window=0, slopes=None, prefix=None, **kw):
    attn = m.Attention(q.shape[1], scale, softcap=softcap, window=window, slopes=slopes)
    off = None if new is None else offsets(new)
    return m.moe_attn_cache(attn, paged.cache, q, paged.table.cuda(), i32(paged.lens), q_offsets=off,
                            prefix=None if prefix is None else i32(prefix), **kw)


def run(lens, new, heads, kv, dim, page, dtype, softcap=0.0, window=0, slopes=False, prefix=None,
        seed=0, grow=1.0):
    paged = ref.Paged(lens, kv, dim, page, seed, dtype=dtype, grow=grow)
    rows = len(lens) if new is None else sum(new)
    q = queries(rows, heads, dim, dtype)
    sl = (0.5 ** torch.linspace(1, 8, heads)).cuda() if slopes else None
    scale = float(np.float32(dim ** -0.5))
    out = call(paged, q, new, scale, softcap, window, sl, prefix)
    ref.check_batch(out, paged, q, new or [1] * len(lens), dtype, scale, softcap, sl, prefix, window)
    return paged, q, out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 255, 257, 600])
def test_one_token(n, dim, dtype):
    run([n], None, 8, 2, dim, 16, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (16, 1), (17, 1), (40, 1), (5, 5), (14, 2), (24, 8),
                                      (128, 1)])
def test_head_layouts(heads, kv, dtype):
    run([77, 300, 5], None, heads, kv, 64, 32, dtype)
    run([77, 300, 5], [4, 2, 5], heads, kv, 64, 32, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages(page, dtype):
    run([1, page, page + 1, 3 * page - 1, 500], [1, 3, page, 7, 2], 6, 2, 128, page, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 5, 33, 130, 300])
def test_rows_of_a_sequence(new, dim, dtype):
    run([300], [new], 4, 2, dim, 16, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_mixed_batch(dtype):
    """Chunks, single and drafted tokens, requests without rows or without tokens."""
    run([400, 90, 0, 33, 1000, 7], [200, 1, 1, 0, 4, 7], 6, 2, 128, 16, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 200, 10**9])
def test_windows(window, dtype):
    run([500, 64, 1], [130, 1, 1], 4, 2, 64, 32, dtype, window=window)
    run([500, 64, 1], None, 4, 2, 64, 32, dtype, window=window)


@pytest.mark.parametrize("dtype", TYPES)
def test_prefixes(dtype):
    """Prefixes that end before, within and after the rows; longer than the text (no mask at all)."""
    run([300, 300, 300, 90, 10], [80, 80, 80, 90, 1], 4, 2, 64, 16, dtype, prefix=[10, 250, 1000, 90, 0])
    run([300, 300], [80, 80], 4, 2, 64, 16, dtype, prefix=[260, 33], window=50)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("grow", [0.1, 1.0, 8.0])
def test_capped_scores(grow, dtype):
    """Scores from where the tanh is a line to where it is flat."""
    run([200, 40], [50, 1], 4, 2, 64, 16, dtype, softcap=5.0, grow=grow)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cap", [1e-39, 70.0, 1e4, 1e30, 3e38])
def test_caps_far_from_the_scores(cap, dtype):
    """Caps that hardly bend the scores (where a tanh times its cap loses what is small against it),
    that bend some, and one below the normal numbers, under which all tokens weigh the same."""
    run([300, 40], [130, 1], 4, 2, 64, 16, dtype, softcap=float(np.float32(cap)), grow=8.0)
    run([300, 40], None, 4, 2, 128, 16, dtype, softcap=float(np.float32(cap)), grow=8.0)
    run([300], [100], 4, 2, 64, 16, dtype, softcap=float(np.float32(cap)), grow=8.0, slopes=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_bias_by_distance(dtype):
    run([200, 700], [50, 3], 6, 2, 64, 16, dtype, slopes=True)
    run([200, 700], [50, 3], 6, 2, 64, 16, dtype, slopes=True, softcap=20.0, window=100,
        prefix=[180, 0])


@pytest.mark.parametrize("dtype", TYPES)
def test_long_sequences_are_cut(dtype):
    """One long text and a short one: pieces of the long one are joined."""
    run([20001, 40], None, 4, 1, 64, 64, dtype)
    run([9001, 2000], [3, 20], 4, 1, 128, 128, dtype)


def test_f32_holds_f32():
    """The error's size over many outputs, not its bound: independent roundings add as squares.
    Scores of D exact products, about sqrt(D) half steps of their largest partial sums (|s| < 8
    here), act on a weight directly; with the rest an output is within 2^-24 (8 sqrt(D) + 8
    sqrt(n / 8)) of its size in the mean.  (16 bits of q or of the weights would be 2^-17.)"""
    D, n = 128, 1000
    paged = ref.Paged([n], 2, D, 64, 3)
    q = queries(64, 8, D, torch.float32)
    scale = float(np.float32(D ** -0.5))
    out = ref.f64(call(paged, q, [64], scale))
    want, _, _ = ref.attention(ref.f64(q), *paged.values(0), scale)
    off = np.linalg.norm(out - want) / np.linalg.norm(want)
    assert off < 2.0**-24 * (8 * D**0.5 + 8 * (n / 8)**0.5) < 2.0**-16
    assert off < 1e-6


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_what_masked_places_hold(dim, dtype):
    """NaN blocks in keys and values where no row sees them change nothing; where rows see them,
    just those rows (keys) and just the block's channels of those rows (values) are NaN."""
    n, new = 150, 40
    paged = ref.Paged([n], 2, dim, 16, 4, dtype=dtype)
    q = queries(new, 4, dim, dtype)
    scale = float(np.float32(dim ** -0.5))
    clean = call(paged, q, [new], scale)
    # rows are at 110 .. 149; a window of 20: token 80 is seen by none, 129 by rows 129 .. 148
    paged.k[0][80, 0, 3] = float("nan")
    paged.v[0][80, 1, dim - 1] = float("inf")
    paged.v[0][129, 0, 33] = -float("inf")
    paged.k[0][139, 1, 0] = float("nan")
    m.moe_kv_write(paged.cache, paged.k[0].cuda(), paged.v[0].cuda(), paged.slots[0].cuda())
    out = call(paged, q, [new], scale, window=20)
    ref.check_batch(out, paged, q, [new], dtype, scale, window=20)
    bad = torch.isnan(out)
    assert bad[19:39, 0:2, 32:64].all() and not bad[:19].any() and not bad[19:29, 2:4].any()
    assert bad[29:, 2:4].all() and not bad[39, 0:2].any() and not bad[:, 0:2, :32].any()
    # without a window the rows see all of them
    out = call(paged, q, [new], scale)
    ref.check_batch(out, paged, q, [new], dtype, scale)
    # and a single row, which the waves of a workgroup share
    out = call(paged, q[-1:], [1], scale, window=11)
    ref.check_batch(out, paged, q[-1:], [1], dtype, scale, window=11)
    assert not torch.isnan(clean).any()


@pytest.mark.parametrize("dtype", TYPES)
def test_infinite_and_nan_rows(dtype):
    """A row that is no number stays one, alone."""
    paged = ref.Paged([90], 1, 64, 16, 5, dtype=dtype)
    q = queries(4, 2, 64, dtype)
    clean = call(paged, q, [4], 0.125)
    q2 = q.clone()
    q2[1, 0, 7] = float("nan")
    q2[2, 1, 9] = float("inf")
    out = call(paged, q2, [4], 0.125)
    bad = torch.isnan(out).any(-1)
    assert bad[1, 0] and bad[2, 1] and int(bad.sum()) == 2
    keep = ~bad
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("dtype", TYPES)
def test_very_large_and_very_small(dtype):
    """Scores far apart (weights of 0 and 1), keys and values at the ends of the scales."""
    paged = ref.Paged([130], 2, 64, 16, 6, dtype=dtype, grow=1e4)
    paged.v[0] *= 1e30
    m.moe_kv_write(paged.cache, paged.k[0].cuda(), paged.v[0].cuda(), paged.slots[0].cuda())
    q = queries(20, 4, 64, dtype)
    out = call(paged, q, [20], 1.0)
    k, v = paged.values(0)
    want, size, _ = ref.attention(ref.f64(q), k, v, 1.0)
    # rows whose two best keys are closer than the scores' own error are left to the other tests
    s = np.einsum("rhd,jhd->rhj", ref.f64(q), np.repeat(k, 2, axis=1))
    ok = ref.sees(130, 20)[:, None, :] & np.ones((20, 4, 1), dtype=bool)
    s = np.sort(np.where(ok, s, -np.inf), axis=2)
    sure = s[:, :, -1] - s[:, :, -2] > 40
    assert sure.mean() > 0.9
    got = ref.f64(out)
    # Both sides differ from the best token's value by the other weights times values: 129 weights of
    # at most e^-40 each, in the kernel times e^d for scores that are off by d = (D + 16) 2^-24 of the
    # products' magnitudes, 64 of 1e4 |q| |k| with a mean of 0.64: 4.1e5, so d < 2 and e^d < 8.  So
    # 129 (1 + 8) e^-40 = 5e-15 of the largest value.
    atol = 129 * 9 * np.exp(-40) * np.abs(v).max()
    assert np.allclose(got[sure], want[sure], rtol=2 * ref.half_step(dtype), atol=atol)
    assert np.isfinite(got).all()


def test_rows_behind_the_last_sequence_are_left():
    paged = ref.Paged([100, 40], 1, 64, 16, 7)
    q = queries(9, 2, 64, torch.float32)
    out = torch.full_like(q, 7.0)
    call(paged, q, [3, 2], 0.125, out=out)
    ref.check_batch(out[:5], paged, q, [3, 2], torch.float32, 0.125)
    assert (out[5:] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(dtype):
    """Queries as part of a fused projection at odd addresses, heads before rows in the output, a
    table that is part of a larger one."""
    lens, new = [70, 33], [6, 1]
    paged = ref.Paged(lens, 2, 64, 16, 8, dtype=dtype)
    fused = queries(7, 1, 4 * 64 + 5, dtype)[:, 0]
    q = fused[:, 3: 3 + 256].view(7, 4, 64)
    out = torch.empty((4, 7, 64), dtype=dtype, device="cuda").transpose(0, 1)
    wide = torch.full((2, paged.table.shape[1] + 9), -5, dtype=torch.int32, device="cuda")
    wide[:, 2: 2 + paged.table.shape[1]] = paged.table.cuda()
    attn = m.Attention(4, 0.125)
    m.moe_attn_cache(attn, paged.cache, q, wide[:, 2: 2 + paged.table.shape[1]], i32(lens),
                     q_offsets=offsets(new), out=out)
    ref.check_batch(out, paged, q, new, dtype, 0.125)


def test_lengths_and_offsets_out_of_range_are_kept_in_it():
    """Lengths past the table, negative ones, offsets past the rows or going back: nothing outside the
    arguments is touched, and the sequences that are right are right."""
    lens = [64, 50]
    paged = ref.Paged(lens, 1, 64, 16, 9, wide=4)
    paged.table[1, 3:] = paged.table[1, 3]
    q = queries(4, 2, 64, torch.float32)
    attn = m.Attention(2, 0.125)
    table = paged.table.cuda()

    def go(lens, off):
        out = torch.full_like(q, 3.0)
        m.moe_attn_cache(attn, paged.cache, q, table, i32(lens), q_offsets=i32(off), out=out)
        return out
    good = go(lens, [0, 2, 4])
    assert torch.equal(go([10**9, 50], [0, 2, 4]), good)          # (the first has 4 pages of 16)
    assert torch.equal(go([64, 50], [0, 2, 99]), good)
    out = go([-5, 50], [0, 2, 4])
    assert not out[:2].any() and torch.equal(out[2:], good[2:])
    out = go([64, 50], [0, 4, 2])                                 # the second has none
    assert torch.isfinite(out).all()
    out = go([64, 50], [-3, 2, 4])
    assert torch.equal(out[2:], good[2:])
    go([64, 50], [0, 4, 0])


def test_pages_that_are_none_read_as_nan():
    paged = ref.Paged([64, 40], 1, 64, 16, 10)
    q = queries(5, 2, 64, torch.bfloat16)
    good = call(paged, q, [4, 1], 0.125)
    for bad in (-1, 10**6, 2**31 - 1, -2**31):
        keep = int(paged.table[0, 1])
        paged.table[0, 1] = bad
        out = call(paged, q, [4, 1], 0.125)
        assert torch.isnan(out[:4]).all() and torch.equal(out[4:], good[4:])
        # masked, it is not missed
        out = call(paged, q, [4, 1], 0.125, window=20)
        assert torch.isfinite(out).all()
        paged.table[0, 1] = keep


def test_a_call_without_rows_or_sequences():
    paged = ref.Paged([10], 1, 64, 16, 11)
    attn = m.Attention(2, 0.125)
    none = torch.empty((0, 2, 64), device="cuda")
    out = m.moe_attn_cache(attn, paged.cache, none, paged.table.cuda(), i32([10]),
                           q_offsets=i32([0, 0]))
    assert out.shape == (0, 2, 64)
    table = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    out = m.moe_attn_cache(attn, paged.cache, none, table, i32([]))
    assert out.shape == (0, 2, 64)
    # a table without pages: no token to see
    q = queries(1, 2, 64, torch.float32)
    out = m.moe_attn_cache(attn, paged.cache, q, torch.empty((1, 0), dtype=torch.int32, device="cuda"),
                           i32([5]))
    assert not out.any()


def test_many_sequences():
    """More sequences than a wave looks at in one step, cut and not."""
    lens = [1 + 7 * i % 90 for i in range(150)]
    run(lens, None, 2, 1, 64, 16, torch.bfloat16)
    new = [min(n, i % 4) for i, n in enumerate(lens)]
    run(lens, new, 2, 1, 64, 16, torch.bfloat16)
    run([5000] + lens, [1] + new, 2, 1, 64, 16, torch.float32)
    lens = [1 + 7 * i % 40 for i in range(700)]
    run(lens, [min(n, i % 3) for i, n in enumerate(lens)], 4, 2, 64, 16, torch.bfloat16)


def test_one_workspace_for_every_batch():
    """The size for the largest batch serves each smaller one, whatever is in it."""
    paged = ref.Paged([3000, 2000, 800, 64], 2, 128, 64, 12)
    attn = m.Attention(8, 0.1)
    table, lens = paged.table.cuda(), i32(paged.lens)
    n = m.moe_attn_cache_workspace_bytes(attn, paged.cache, 4000, 4)
    last = 0
    for rows in (1, 4, 16, 64, 300, 1000, 4000):
        have = m.moe_attn_cache_workspace_bytes(attn, paged.cache, rows, 4)
        assert last <= have <= n
        last = have
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    for new in ([1, 1, 1, 1], [9, 1, 0, 3], [100, 64, 3, 64], [2000, 1, 1, 1]):
        q = queries(sum(new), 8, 128, torch.bfloat16)
        got = m.moe_attn_cache(attn, paged.cache, q, table, lens, q_offsets=offsets(new), ws=ws)
        want = m.moe_attn_cache(attn, paged.cache, q, table, lens, q_offsets=offsets(new))
        assert torch.equal(got, want)
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("new", [None, [3, 40]])
def test_streams_and_replays_with_other_lengths(new):
    """A captured call replays with other queries, lengths and pages, and equals the eager call bit
    for bit; two graphs share a workspace."""
    paged = ref.Paged([2100, 900], 2, 128, 64, 13)
    rows = 2 if new is None else sum(new)
    q = queries(rows, 8, 128, torch.bfloat16)
    attn = m.Attention(8, 0.1, softcap=30.0)
    table, lens = paged.table.cuda(), i32(paged.lens)
    off = None if new is None else offsets(new)
    ws = torch.empty(m.moe_attn_cache_workspace_bytes(attn, paged.cache, rows, 2), dtype=torch.uint8,
                     device="cuda")
    graphs = []
    for _ in range(2):
        out = torch.empty_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.moe_attn_cache(attn, paged.cache, q, table, lens, q_offsets=off, out=out, ws=ws)
        graphs.append((graph, out))
    for i, n in enumerate(([2100, 900], [64, 1], [1999, 0], [0, 800], [2100, 900])):
        q.copy_(queries(rows, 8, 128, torch.bfloat16, seed=i))
        lens.copy_(i32(n))
        for graph, out in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = m.moe_attn_cache(attn, paged.cache, q, table, lens, q_offsets=off)
        assert torch.equal(graphs[0][1], want) and torch.equal(graphs[1][1], want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.moe_attn_cache(attn, paged.cache, q, table, lens, q_offsets=off, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_a_call_is_the_same_each_time():
    paged, q, out = run([5000, 300], [2, 3], 8, 2, 128, 64, torch.bfloat16)
    for _ in range(3):
        assert torch.equal(call(paged, q, [2, 3], float(np.float32(128 ** -0.5))), out)


def test_refused_in_the_binding():
    paged = ref.Paged([40], 2, 64, 16, 14)
    q, table, lens = queries(1, 4, 64, torch.float32), paged.table.cuda(), i32([40])
    attn = m.Attention(4, 0.125)
    with pytest.raises(TypeError):
        m.moe_attn_cache(attn, paged.cache, q.half(), table, lens)
    with pytest.raises(ValueError):
        m.moe_attn_cache(attn, paged.cache, q.cpu(), table, lens)
    with pytest.raises(ValueError):
        m.moe_attn_cache(attn, paged.cache, q, table, lens.cpu())
    with pytest.raises(TypeError):
        m.moe_attn_cache(attn, paged.cache, q, table.long(), lens)
    with pytest.raises(ValueError):
        m.moe_attn_cache(attn, paged.cache, q[:, :3], table, lens)
    with pytest.raises(m.MoeError):                 # in place
        m.moe_attn_cache(attn, paged.cache, q, table, lens, out=q)
    with pytest.raises(m.MoeError):                 # 2 rows for 1 sequence
        m.moe_attn_cache(attn, paged.cache, queries(2, 4, 64, torch.float32), table, lens)
    with pytest.raises(m.MoeError):                 # 3 query heads for 2 key heads
        m.moe_attn_cache(m.Attention(3, 0.125), paged.cache, q[:, :3].contiguous(), table, lens)


# ------------------------------------------------- the forms for many rows and long texts
@pytest.mark.parametrize("dim,kv,heads,rows,n", [(64, 8, 32, 2048, 2100), (128, 8, 32, 2048, 2100),
                                                 (64, 32, 32, 1030, 1200)])
def test_workgroups_of_256_rows(dim, kv, heads, rows, n):
    """Enough tiles of 256 rows for every CU; some of the rows against the 64-bit form."""
    dtype, page = torch.bfloat16, 32
    paged = ref.Paged([n, 70], kv, dim, page, 20, dtype=dtype)
    q = queries(rows + 1, heads, dim, dtype)
    scale = float(np.float32(dim ** -0.5))
    out = call(paged, q, [rows, 1], scale, window=900)
    k, v = paged.values(0)
    some = [0, 1, 63, 64, 65, rows // 2, rows - 2, rows - 1]
    for r in some:
        last = n - rows + r + 1
        want, size, ds = ref.attention(ref.f64(q[r: r + 1]), k[:last], v[:last], scale, window=900)
        ref.check(out[r: r + 1], want, ref.attention_error(size, ds, last, dtype), dtype)
    ref.check_batch(out[rows:], _only(paged, 1), q[rows:], [1], dtype, scale, window=900)


def _only(paged, s):
    class One:
        lens = [paged.lens[s]]

        @staticmethod
        def values(_):
            return paged.values(s)
    return One


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,n", [(1100, 1100), (1100, 1301)])
def test_more_tiles_than_cus(rows, n, dim):
    """Tiles of 128 rows that leave no CU idle, and are too few for those of 256."""
    run([n], [rows], 32, 32, dim, 64, torch.bfloat16, window=150)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [257, 319, 321, 383, 385, 400, 513])
def test_two_waves_for_the_same_rows(n, dim):
    """Few tiles: a stage's 128 tokens in two halves, of which one may be empty for a row, a wave or
    all; from the text's start and behind a window."""
    run([n], [70], 4, 2, dim, 16, torch.bfloat16)
    run([n, 70, 127, 129, 200], [70, 70, 100, 65, 33], 4, 2, dim, 16, torch.bfloat16)
    run([n, 5], [70, 3], 8, 2, dim, 32, torch.bfloat16, window=40, prefix=[90, 0], softcap=8.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows_over_a_long_text_are_cut(dtype):
    """Tiles of many rows whose tokens are cut and joined (a wave for each row's head); the heads'
    group does not divide a tile, so that a row's heads lie in two."""
    run([3000, 40], [300, 40], 7, 1, 64, 64, dtype)
    run([2600], [110], 24, 1, 128, 64, dtype, window=2500, softcap=20.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [3, 90])
def test_nan_blocks_and_bad_pages_in_cut_calls(new, dtype):
    """NaN keys, NaN values and a page that is none, in a text that is cut, for few and many rows."""
    n, heads = 4000, 4
    paged = ref.Paged([n], 1, 64, 16, 21, dtype=dtype)
    paged.v[0][1000, 0, 40] = float("nan")
    paged.k[0][n - new + 1, 0, 2] = float("nan")
    m.moe_kv_write(paged.cache, paged.k[0].cuda(), paged.v[0].cuda(), paged.slots[0].cuda())
    q = queries(new, heads, 64, dtype)
    out = call(paged, q, [new], 0.125)
    ref.check_batch(out, paged, q, [new], dtype, 0.125)
    bad = torch.isnan(out)
    assert bad[0, :, 32:].all() and not bad[0, :, :32].any() and bad[1:].all()
    paged.table[0, 5] = -7                       # tokens 80 .. 95
    out = call(paged, q, [new], 0.125)
    assert torch.isnan(out).all()
    out = call(paged, q, [new], 0.125, window=n - 200)   # (sees 1000 and not 95)
    assert torch.equal(torch.isnan(out), bad)


@pytest.mark.parametrize("dtype", TYPES)
def test_out_of_range_lengths_with_many_rows(dtype):
    lens = [256, 200]
    paged = ref.Paged(lens, 1, 64, 16, 22, wide=16, dtype=dtype)
    q = queries(160, 2, 64, dtype)
    attn = m.Attention(2, 0.125)
    table = paged.table.cuda()

    def go(lens, off):
        out = torch.full_like(q, 3.0)
        m.moe_attn_cache(attn, paged.cache, q, table, i32(lens), q_offsets=i32(off), out=out)
        return out
    good = go(lens, [0, 80, 160])
    ref.check_batch(good, paged, q, [80, 80], dtype, 0.125)
    assert torch.equal(go([10**9, 200], [0, 80, 160]), good)
    assert torch.equal(go(lens, [0, 80, 10**6]), good)
    out = go([-1, 200], [0, 80, 160])
    assert not out[:80].any() and torch.equal(out[80:], good[80:])
    for off in ([0, 160, 80], [160, 0, 160], [80, 80, 20], [-9, -3, 0]):
        go(lens, off)
    # a row whose place is below 0 sees nothing
    out = go([30, 200], [0, 80, 160])
    assert not out[:50].any() and out[50:80].any()


def test_a_cache_past_4_gib():
    """Pages at both ends of a cache of more than 4 GiB, for few and many rows."""
    kv, dim, page = 32, 128, 256
    per = kv * page * (dim + dim // 16)
    n_pages = 2**32 // per + 5
    cache = m.KVCache(n_pages, page, kv, dim)
    g = torch.Generator().manual_seed(3)
    pages = torch.tensor([n_pages - 1, 0, n_pages - 3], dtype=torch.int32)
    n = 600
    t = torch.arange(n)
    slots = (pages.long()[t // page] * page + t % page).int().cuda()
    k, v = torch.randn(2, n, kv, dim, generator=g).bfloat16()
    m.moe_kv_write(cache, k.cuda(), v.cuda(), slots)
    kk, vv = ref.stored(ref.f64(k)), ref.stored(ref.f64(v))
    scale = float(np.float32(dim ** -0.5))
    attn = m.Attention(kv, scale)
    for new in (1, 80):
        q = queries(new, kv, dim, torch.bfloat16)
        out = m.moe_attn_cache(attn, cache, q, pages.cuda()[None], i32([n]), q_offsets=i32([0, new]))
        want, size, ds = ref.attention(ref.f64(q), kk, vv, scale)
        ref.check(out, want, ref.attention_error(size, ds, n, torch.bfloat16), torch.bfloat16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_scales_that_are_not_positive(scale, dtype):
    scale = float(np.float32(scale))
    paged = ref.Paged([200], 1, 64, 16, 23, dtype=dtype)
    for new in (2, 100):
        q = queries(new, 2, 64, dtype)
        ref.check_batch(call(paged, q, [new], scale), paged, q, [new], dtype, scale)


@pytest.mark.parametrize("dtype", TYPES)
def test_scores_that_grow_along_the_text(dtype):
    """Each stretch of tokens outweighs all before it, and then falls: bases are raised again and
    again, and what came before leaves the sums."""
    n, dim = 700, 64
    paged = ref.Paged([n], 1, dim, 16, 24, dtype=dtype)
    t = torch.arange(n)
    height = 3.0 * torch.floor(t / 16) * (t < 500) - 40.0 * (t >= 500)
    paged.k[0][:, 0, :32] = (height[:, None] / 8).to(dtype)
    m.moe_kv_write(paged.cache, paged.k[0].cuda(), paged.v[0].cuda(), paged.slots[0].cuda())
    for new in (1, 5, 120):
        q = queries(new, 2, dim, dtype)
        q[:, :, :32] = 0.5
        ref.check_batch(call(paged, q, [new], 1.0), paged, q, [new], dtype, 1.0)
