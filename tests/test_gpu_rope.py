"""Rotary positions against their 64-bit form: types, head layouts, odd sizes, axes, far and
negative positions, in place and copied channels, strides, streams and replays."""
import numpy as np
import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")

TYPES = [torch.float32, torch.bfloat16]


def make(rows, heads, dim, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, heads, dim, generator=g).to(dtype).cuda()


def places(rows, axes, seed=0, far=1 << 20):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, far, (axes, rows), generator=g, dtype=torch.int32).cuda()


def compare(got, x, pos, freq, axes=None, interleaved=False, scale=1.0):
    xs, ps = ref.f64(x), pos.cpu().numpy().astype(np.float64).reshape(-1, x.shape[0])
    scale = float(np.float32(scale))
    want = ref.rope(xs, ps, freq, axes, interleaved, scale)
    # (the 64-bit form's own angle: a product's rounding, half of 2^-52 of it, twice for cos and sin)
    far = np.abs(ps).max() * max(freq) * 2.0**-52
    err = ref.rope_error(xs, freq, interleaved, scale) * (1 + far * 2.0**24)
    ref.check(got, want, err, x.dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,dim,rot", [
    (1, 1, 2, 2), (1, 40, 128, 128), (3, 7, 64, 48), (17, 5, 80, 20), (33, 3, 65, 34),
    (2, 9, 129, 18), (700, 12, 128, 128), (5, 2, 1024, 1024), (4000, 24, 64, 64)])
def test_shapes(rows, heads, dim, rot, interleaved, dtype):
    x, freq = make(rows, heads, dim, dtype), ref.frequencies(rot // 2)
    pos = places(rows, 1)[0]
    r = m.Rope(freq, interleaved=interleaved)
    got = m.moe_rope(r, x, pos)
    compare(got, x, pos, freq, interleaved=interleaved)
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", TYPES)
def test_axes(dtype):
    rows, n = 50, 24
    x, freq, axes = make(rows, 6, 64, dtype), ref.frequencies(n), [0, 1, 2] * 8
    pos = places(rows, 3, far=5000)
    r = m.Rope(freq, axes=axes, scale=0.75)
    compare(m.moe_rope(r, x, pos), x, pos, freq, axes, scale=0.75)
    # sections side by side, positions as rows of a larger tensor
    axes = [0] * 4 + [2] * 12 + [1] * 8
    wide = torch.zeros((3, 77), dtype=torch.int32, device="cuda")
    wide[:, :rows] = pos
    r = m.Rope(torch.tensor(freq, dtype=torch.float64), axes=torch.tensor(axes))
    compare(m.moe_rope(r, x, wide[:, :rows]), x, pos, freq, axes)


def test_far_and_negative_positions():
    """Angles of up to 2^31 radians: the fraction of a turn is exact in whole numbers.  The 64-bit
    form takes it from the same product in exact arithmetic."""
    from fractions import Fraction
    at = [0, 1, -1, 2**20 + 1, 10**8 + 7, 2**31 - 1, -2**31, 123456789]
    freq = [1.0, 0.1, 10000.0 ** -0.5, 3.0, 1e-9]
    pi = Fraction(31415926535897932384626433832795028841971, 10**40)
    x = make(len(at), 2, 10, torch.float32)
    pos = torch.tensor(at, dtype=torch.int32, device="cuda")
    got = ref.f64(m.moe_rope(m.Rope(freq), x, pos))
    angle = np.array([[float(Fraction(f) * p % (2 * pi)) for f in freq] for p in at])
    xs = ref.f64(x)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = xs[:, :, :5], xs[:, :, 5:]
    want = np.concatenate([a * c - b * s, b * c + a * s], axis=2)
    assert (np.abs(got - want) <= ref.rope_error(xs, freq, False, 1.0) + 2.0**-24 * np.abs(want)).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_in_place(dtype):
    """Query and key heads of a fused projection, heads before rows, rows at odd addresses."""
    rows, dim, freq = 19, 64, ref.frequencies(32)
    pos = places(rows, 1)[0]
    r = m.Rope(freq)
    fused = make(rows, 1, 12 * dim + 3, dtype)[:, 0]
    before = fused.clone()
    part = fused[:, 3: 3 + 9 * dim].view(rows, 9, dim)
    x = part.clone()
    assert m.moe_rope(r, part, pos, out=part) is part
    compare(part, x, pos, freq)
    assert torch.equal(fused[:, :3], before[:, :3])
    assert torch.equal(fused[:, 3 + 9 * dim:], before[:, 3 + 9 * dim:])
    swapped = make(8, rows, dim, dtype).transpose(0, 1)
    out = torch.empty((8, rows, dim), dtype=dtype, device="cuda").transpose(0, 1)
    compare(m.moe_rope(r, swapped, pos, out=out), swapped, pos, freq)


def test_partial_rotation_in_place_leaves_the_rest():
    x = make(5, 3, 40, torch.bfloat16)
    y = x.clone()
    m.moe_rope(m.Rope(ref.frequencies(6)), y, places(5, 1)[0], out=y)
    compare(y, x, places(5, 1)[0], ref.frequencies(6))


def test_a_head_does_not_depend_on_its_call():
    x, freq = make(4096, 40, 128, torch.bfloat16), ref.frequencies(64)
    pos = places(4096, 1)[0]
    r = m.Rope(freq)
    whole = m.moe_rope(r, x, pos)
    for row, head in ((0, 0), (1, 39), (4095, 17)):
        one = x[row: row + 1, head: head + 1]
        assert torch.equal(m.moe_rope(r, one, pos[row: row + 1]), whole[row: row + 1, head: head + 1])


def test_nothing_to_do_and_not_numbers():
    r = m.Rope([1.0, 0.5])
    none = torch.empty((0, 3, 4), device="cuda")
    assert m.moe_rope(r, none, torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 3, 4)
    x = torch.ones((2, 1, 4), device="cuda")
    x[0, 0, 1] = float("nan")
    y = m.moe_rope(r, x, torch.tensor([1, 1], dtype=torch.int32, device="cuda"))
    assert torch.isnan(y[0, 0]).tolist() == [False, True, False, True]
    assert torch.isfinite(y[1]).all()


def test_streams_and_replays():
    x, freq, pos = make(9, 4, 64, torch.float32), ref.frequencies(32), places(9, 1)[0]
    r = m.Rope(freq)
    want = m.moe_rope(r, x, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.moe_rope(r, x, pos, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        m.moe_rope(r, x, pos, out=out)
    for i in range(4):
        pos.copy_(places(9, 1, seed=i)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, m.moe_rope(r, x, pos))
