"""Forms of the kernels around the 4-bit cache that only certain sizes reach: heads of 256 cut and joined
and with 17 to 64 (token, head) pairs, cut calls in tiles of 128 rows, several rows a thread in the
cache's writing and reading, groups of heads a thread that do not divide the heads in the rotary
positions."""
import pytest
import torch

import attn_ref as ref
from test_gpu_attn import TYPES, call, i32, queries, run
from test_gpu_kv_cache import same
from test_gpu_rope import compare, make, places

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [200, 900, 5000])
@pytest.mark.parametrize("new,heads", [(1, 17), (5, 4), (5, 6), (8, 8)])
def test_17_to_64_pairs(new, heads, n, dim, dtype):
    """Texts below 256 tokens, of up to 1024 and ones that are cut."""
    run([n, 33], [new, 2], heads, 1, dim, 32, dtype)
    run([n], [new], heads, 1, dim, 64, dtype, window=n - 50, softcap=20.0, slopes=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [128, 256])
def test_cut_calls(dim, dtype):
    """Few rows and many, joined by one wave a row's head and by four."""
    run([20001, 40], None, 4, 1, dim, 64, dtype)
    run([9001, 2000], [3, 20], 4, 2, dim, 128, dtype)
    run([3000, 40], [300, 40], 7, 1, dim, 64, dtype)
    run([2600], [110], 24, 1, dim, 64, dtype, window=2500, softcap=20.0)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,heads", [(100, 1), (65, 1), (25, 4), (128, 1)])
def test_cut_calls_in_tiles_of_128_rows(new, heads, dim):
    run([4001], [new], heads, 1, dim, 64, torch.bfloat16)
    run([4001], [new], heads, 1, dim, 64, torch.bfloat16, window=3900, prefix=[500])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("new", [3, 10, 90])
def test_nan_blocks_and_bad_pages_in_cut_calls(new, dim, dtype):
    n, heads = 4000, 4
    paged = ref.Paged([n], 1, dim, 16, 42, dtype=dtype)
    paged.v[0][1000, 0, dim - 24] = float("nan")
    paged.k[0][n - new + 1, 0, 2] = float("nan")
    m.moe_kv_write(paged.cache, paged.k[0].cuda(), paged.v[0].cuda(), paged.slots[0].cuda())
    q = queries(new, heads, dim, dtype)
    out = call(paged, q, [new], 0.125)
    ref.check_batch(out, paged, q, [new], dtype, 0.125)
    bad = torch.isnan(out)
    assert bad[0, :, dim - 32:].all() and not bad[0, :, :dim - 32].any() and bad[1:].all()
    paged.table[0, 5] = -7                       # tokens 80 .. 95
    assert torch.isnan(call(paged, q, [new], 0.125)).all()
    out = call(paged, q, [new], 0.125, window=n - 200)   # (sees 1000 and not 95)
    assert torch.equal(torch.isnan(out), bad)


# (rows of 2 heads dim / 8 threads, at most 256; four a thread from 512 workgroups on)
MANY = [(32771, 1, 64), (8197, 3, 64), (2053, 8, 128), (4103, 5, 64), (2050, 5, 256), (8193, 1, 256)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,heads,dim", MANY)
def test_four_rows_a_thread(rows, heads, dim, dtype):
    """Every row written and read back, among rows without a slot; the cache's other bytes are left."""
    g = torch.Generator().manual_seed(rows)
    k = (3 * torch.randn(rows, heads, dim, generator=g)).to(dtype)
    v = torch.randn(rows, heads, dim, generator=g).to(dtype)
    page = 64
    cache = m.KVCache(rows // page + 4, page, heads, dim)
    slots = torch.randperm(cache.n_pages * page, generator=g)[:rows].int()
    none = torch.rand(rows, generator=g) < 0.01
    none[-1] = True
    slots[none] = -1
    slots = slots.cuda()
    m.moe_kv_write(cache, k.cuda(), v.cuda(), slots)
    few = m.KVCache(cache.n_pages, page, heads, dim)     # the same by calls of few rows
    for at in range(0, rows, 1500):
        m.moe_kv_write(few, k[at: at + 1500].cuda(), v[at: at + 1500].cuda(), slots[at: at + 1500])
    assert torch.equal(cache.tensors[0], few.tensors[0])
    wk, wv = ref.stored(ref.f64(k)), ref.stored(ref.f64(v))
    wk[none], wv[none] = 0, 0
    for out in TYPES:
        gk, gv = m.moe_kv_read(cache, slots, dtype=out)
        same(gk, wk, out)
        same(gv, wv, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,heads,dim", [(8197, 3, 64), (2053, 8, 128), (2050, 5, 256)])
def test_four_rows_a_thread_at_odd_addresses(rows, heads, dim, dtype):
    """Slices of a fused projection whose rows have their elements' alignment alone, heads before
    rows; what lies beside them is left."""
    n = heads * dim
    fused = torch.randn(rows, 3 * n + 1, device="cuda").to(dtype)
    k, v = fused[:, 1: 1 + n].view(rows, heads, dim), fused[:, 1 + 2 * n:].view(rows, heads, dim)
    cache = m.KVCache(rows // 32 + 1, 32, heads, dim)
    slots = i32(torch.randperm(cache.n_pages * 32)[:rows])
    m.moe_kv_write(cache, k, v, slots)
    out = torch.full((rows, 2 * n + 1), 7.0, dtype=dtype, device="cuda")
    ko = out[:, 1: 1 + n].view(rows, heads, dim)
    vo = torch.zeros(heads, rows, dim, dtype=dtype, device="cuda").transpose(0, 1)
    m.moe_kv_read(cache, slots, k=ko, v=vo)
    same(ko, ref.stored(ref.f64(k)), dtype)
    same(vo, ref.stored(ref.f64(v)), dtype)
    assert (out[:, 0] == 7.0).all() and (out[:, 1 + n:] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,dim,rot", [(4000, 25, 64, 64), (2500, 25, 80, 48), (3001, 13, 130, 130),
                                                (9001, 11, 64, 64)])
def test_groups_of_heads_that_do_not_divide_them(rows, heads, dim, rot, interleaved, dtype):
    """2 or 3 heads a thread: the last one of a row has fewer."""
    x, freq, pos = make(rows, heads, dim, dtype), ref.frequencies(rot // 2), places(rows, 1)[0]
    r = m.Rope(freq, interleaved=interleaved)
    got = m.moe_rope(r, x, pos)
    compare(got, x, pos, freq, interleaved=interleaved)
    assert torch.equal(got[..., rot:], x[..., rot:])
    y = x.clone()
    m.moe_rope(r, y, pos, out=y)
    assert torch.equal(y, got)
