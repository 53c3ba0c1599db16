"""The 4-bit cache, bit for bit: every midpoint of the codes, scales at both ends of their range,
blocks that are not numbers, head layouts and pages, rows without a slot, untouched slots."""
import numpy as np
import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")

TYPES = [torch.float32, torch.bfloat16]


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32, device="cuda")


def same(got, want, dtype):
    """Equal values (what the cache holds is exact in both types), NaN with NaN."""
    want = torch.from_numpy(want).to(dtype).cuda()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,page,rows", [(1, 16, 1), (3, 16, 37), (8, 64, 130), (5, 256, 300),
                                             (2, 32, 33), (1, 128, 129)])
def test_round_trip(rows, heads, page, dim, dtype):
    g = torch.Generator().manual_seed(rows)
    shape = (rows, heads, dim)
    k = (torch.randn(shape, generator=g) * torch.exp(3 * torch.randn(rows, heads, 1, generator=g))).to(dtype)
    v = torch.randn(shape, generator=g).to(dtype)
    n_pages = rows // page + 3
    cache = m.KVCache(n_pages, page, heads, dim)
    slots = i32(torch.randperm(n_pages * page, generator=g)[:rows])
    m.moe_kv_write(cache, k.cuda(), v.cuda(), slots)
    for out in TYPES:
        gk, gv = m.moe_kv_read(cache, slots, dtype=out)
        same(gk, ref.stored(ref.f64(k)), out)
        same(gv, ref.stored(ref.f64(v)), out)
    # what the cache holds is written again without change
    before = cache.tensors[0].clone()
    m.moe_kv_write(cache, gk, gv, slots)
    assert torch.equal(cache.tensors[0], before)


@pytest.mark.parametrize("dtype", TYPES)
def test_every_midpoint(dtype):
    """Values on and beside every border between codes, of both signs, at scales from the least to
    the largest."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    eps = torch.finfo(dtype).eps
    near = np.concatenate([borders, borders * (1 - eps), borders * (1 + eps)])
    near = np.concatenate([near, -near])
    rows = []
    for e in (-125, -100, -30, -1, 0, 1, 30, 100, 124):
        for top in (4.0, 6.0, 3.5, 7.0 * (1 - eps)):
            for lo in range(0, len(near), 31):
                b = np.zeros(32)
                b[0] = top
                part = near[lo: lo + 31]
                b[1: 1 + len(part)] = part
                rows.append(b * 2.0**e)
    x = np.array(rows)
    x = x.reshape(-1, 2, 1, 32) if len(x) % 2 == 0 else np.concatenate([x, x[:1]]).reshape(-1, 2, 1, 32)
    x = torch.from_numpy(x.transpose(0, 2, 1, 3).reshape(-1, 1, 64)).to(dtype)
    n = x.shape[0]
    cache = m.KVCache(n // 16 + 1, 16, 1, 64)
    slots = i32(torch.arange(n))
    m.moe_kv_write(cache, x.cuda(), -x.cuda(), slots)
    k, v = m.moe_kv_read(cache, slots, dtype=torch.float32)
    want = ref.stored(ref.f64(x))
    same(k, want, torch.float32)
    same(v, -want, torch.float32)


def test_ends_of_the_range():
    """The largest numbers, numbers below the least scale's step, zeros, infinities and NaN: a
    block that is not all numbers reads as NaN, its neighbours as they are."""
    big = torch.finfo(torch.float32).max
    x = torch.randn(8, 1, 128, generator=torch.Generator().manual_seed(1))
    x[0, 0, 0:32] = big
    x[1, 0, 32:64] = 0.0
    x[1, 0, 33] = -0.0
    x[2, 0, 64:96] = 2.0**-140                 # subnormal: less than half a step of the least scale
    x[3, 0, 5] = float("inf")
    x[4, 0, 127] = float("nan")
    x[5, 0, 0:32] = 2.0**-126 * torch.arange(32)
    x[6, 0, 70] = -float("inf")
    cache = m.KVCache(1, 16, 1, 128)
    slots = i32([3, 0, 15, 7, 8, 1, 12, 5])
    m.moe_kv_write(cache, x.cuda(), x.flip(0).cuda(), slots)
    want = ref.stored(ref.f64(x))
    assert np.isnan(want[3, 0, :32]).all() and np.isfinite(want[3, 0, 32:]).all()
    assert (want[2, 0, 64:96] == 0).all() and want[0, 0, 0] == 6 * 2.0**125
    k, v = m.moe_kv_read(cache, slots, dtype=torch.float32)
    same(k, want, torch.float32)
    same(v, want[::-1].copy(), torch.float32)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_without_a_slot_and_other_slots(dim):
    """Slots below 0 and past the cache: nothing written, zeros read; no byte of another slot
    changes; a slot may be read twice."""
    heads, page, n_pages = 3, 16, 4
    cache = m.KVCache(n_pages, page, heads, dim)
    fill = torch.randn(page * n_pages, heads, dim, device="cuda")
    everything = i32(torch.arange(page * n_pages))
    m.moe_kv_write(cache, fill, 2 * fill, everything)
    bk, bv = m.moe_kv_read(cache, everything, dtype=torch.float32)
    x = torch.randn(6, heads, dim, device="cuda")
    slots = i32([-1, 5, page * n_pages, 2**31 - 1, -2**31, 63])
    m.moe_kv_write(cache, x, 3 * x, slots)
    ak, av = m.moe_kv_read(cache, everything, dtype=torch.float32)
    for a, b, f in ((ak, bk, 1), (av, bv, 3)):
        want = b.clone()
        want[5] = torch.from_numpy(ref.stored(ref.f64(f * x[1])))
        want[63] = torch.from_numpy(ref.stored(ref.f64(f * x[5])))
        assert torch.equal(a, want)
    k, v = m.moe_kv_read(cache, i32([5, -1, 5, 64, 63]), dtype=torch.float32)
    assert torch.equal(k[0], ak[5]) and torch.equal(k[2], ak[5]) and torch.equal(v[4], av[63])
    assert not k[1].any() and not k[3].any() and not v[1].any() and not v[3].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(dtype):
    """Slices of a fused projection at odd addresses; heads before rows."""
    rows, heads, dim = 21, 4, 64
    fused = torch.randn(rows, 3 * heads * dim + 1, device="cuda").to(dtype)
    k = fused[:, 1: 1 + heads * dim].view(rows, heads, dim)
    v = fused[:, 1 + 2 * heads * dim:].view(rows, heads, dim)
    cache = m.KVCache(2, 16, heads, dim)
    slots = i32(torch.randperm(32)[:rows])
    m.moe_kv_write(cache, k, v, slots)
    out = torch.zeros(rows, 2 * heads * dim + 1, dtype=dtype, device="cuda")
    ko = out[:, 1: 1 + heads * dim].view(rows, heads, dim)
    vo = torch.zeros(heads, rows, dim, dtype=dtype, device="cuda").transpose(0, 1)
    m.moe_kv_read(cache, slots, k=ko, v=vo)
    same(ko, ref.stored(ref.f64(k)), dtype)
    same(vo, ref.stored(ref.f64(v)), dtype)
    assert not out[:, 0].any() and not out[:, 1 + heads * dim:].any()


def test_offsets_past_32_bits():
    """A cache of more than 4 GiB: its last slots, and that its first are as they were."""
    heads, dim, page = 64, 256, 256
    per = heads * page * (dim + dim // 16)
    n_pages = (2**32) // per + 3
    cache = m.KVCache(n_pages, page, heads, dim)
    assert cache.tensors[0].numel() > 2**32
    x = torch.randn(4, heads, dim, device="cuda")
    last = n_pages * page - 1
    slots = i32([last, 0, last - page * 2 - 1, last - 1])
    m.moe_kv_write(cache, x, -x, slots)
    k, v = m.moe_kv_read(cache, slots, dtype=torch.float32)
    want = ref.stored(ref.f64(x))
    same(k, want, torch.float32)
    same(v, -want, torch.float32)
    assert int((cache.tensors[0] != 0).sum()) <= 4 * heads * 2 * (dim // 2 + dim // 32)


def test_streams_and_replays():
    cache = m.KVCache(4, 16, 2, 128)
    k, v = torch.randn(2, 3, 2, 128, device="cuda")
    slots = i32([5, 40, -1])
    graph = torch.cuda.CUDAGraph()
    ko, vo = torch.empty(3, 2, 128, device="cuda"), torch.empty(3, 2, 128, device="cuda")
    m.moe_kv_write(cache, k, v, slots)
    with torch.cuda.graph(graph):
        m.moe_kv_write(cache, k, v, slots)
        m.moe_kv_read(cache, slots, k=ko, v=vo)
    for i in range(4):
        k.copy_(torch.randn(3, 2, 128))
        slots.copy_(i32([(7 * i) % 64, 63 - i, -1 if i % 2 else 30]))
        graph.replay()
        torch.cuda.synchronize()
        want = ref.stored(ref.f64(k))
        if i % 2:
            want[2] = 0
        same(ko, want, torch.float32)
        m.moe_kv_read(cache, slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_kv_write(cache, k, v, slots, stream=side)
    sk, _ = m.moe_kv_read(cache, slots, dtype=torch.float32, stream=side)
    side.synchronize()
    assert torch.equal(sk, ko)
