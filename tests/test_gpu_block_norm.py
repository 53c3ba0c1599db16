"""Block norms and the row quantiser against 64-bit forms.

Tolerance.  A row's sum of squares is at most 32 fused steps in a thread, 6
over a wave and 16 over the waves, so its relative error is below 54 2^-24 and
its inverse root's below 27 2^-24; mean, root and the three products add at
most 8 more: |h - ref| <= 40 2^-24 |ref|.  A block's result
b carries that too, and out = rs res + g b at most two roundings of its own:
|out - ref| <= 48 2^-24 (|rs res| + |g b|).  A bf16 result adds half a step,
at most 2^-8 of its value (2^-134 among the subnormals).
"""
import numpy as np
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0**-24


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rows_of(g, rows, cols, dtype, pad=0, scale=1.0, shift=0):
    """A [rows][cols] view whose rows lie cols + pad apart, `shift` elements
    into its buffer."""
    ld = cols + pad
    buf = (scale * torch.randn(rows * ld + shift, generator=g, device=DEV)).to(dtype)
    return buf[shift:].view(rows, ld)[:, :cols]


def close(got, want, mag, units, dtype):
    got = ref.f64(got)
    tol = units * U * mag
    if dtype == BF16:
        tol = tol + 2.0**-8 * np.abs(want) * (1 + units * U) + 2.0**-134
    bad = np.abs(got - want) > tol
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, worst "
                           f"{(np.abs(got - want) / np.maximum(tol, 1e-300)).max():.2f} x tol")


COLS = [1, 7, 8, 31, 64, 100, 512, 1000, 2049, 4096, 4104, 8192, 16384]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("xt,ht", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
def test_pre_matches_formula(cols, xt, ht):
    g = gen(cols)
    w = 1 + 0.2 * torch.randn(cols, generator=g, device=DEV)
    for rows, pad, shift in ((1, 0, 0), (5, 0, 0), (3, 8, 0), (4, 3, 1)):
        x = rows_of(g, rows, cols, xt, pad, 3.0, shift)
        h = m.moe_norm_pre(m.Norm(cols, pre_w=w, eps=1e-5), x, h_dtype=ht)
        want = ref.rms(ref.f64(x), ref.f64(w), float(np.float32(1e-5)))
        close(h, want, np.abs(want), 40, ht)
        h2 = m.moe_norm_pre(m.Norm(cols, eps=1e-5), x, h_dtype=ht)
        want = ref.rms(ref.f64(x), None, float(np.float32(1e-5)))
        close(h2, want, np.abs(want), 40, ht)


GATES = ["none", "number", "channel", "token", "full", "wide"]


def make_gate(g, kind, rows, cols, dtype):
    r = lambda *s: (0.5 + 0.3 * torch.randn(*s, generator=g, device=DEV)).to(dtype)  # noqa: E731
    return {"none": lambda: None, "number": lambda: r(1), "channel": lambda: r(cols),
            "token": lambda: r(rows, 1), "full": lambda: r(rows, cols),
            "wide": lambda: r(rows, cols + 5)[:, :cols]}[kind]()


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("yt,rt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_post_matches_formula(gate, yt, rt):
    for i, (rows, cols, pad) in enumerate([(1, 4096, 0), (3, 100, 0), (6, 64, 8), (2, 2049, 1),
                                           (5, 8200, 0), (7, 1, 0)]):
        g = gen(100 + i)
        w = 1 + 0.2 * torch.randn(cols, generator=g, device=DEV)
        y, res = rows_of(g, rows, cols, yt, pad, 2.0), rows_of(g, rows, cols, rt, pad, 5.0)
        gt = make_gate(g, gate, rows, cols, BF16 if i % 2 else F32)
        for post in (True, False):
            N = m.Norm(cols, post_w=w, post_norm=post, eps=1e-6, residual_scale=0.75)
            out = m.moe_norm_post(N, y, res, gate=gt)
            b = ref.rms(ref.f64(y), ref.f64(w), float(np.float32(1e-6))) if post else ref.f64(y)
            b = b if gt is None else b * ref.f64(gt)
            r = 0.75 * ref.f64(res)
            close(out, r + b, np.abs(r) + np.abs(b), 48, rt)


@pytest.mark.parametrize("rt,ht", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("cols", [32, 96, 2048, 4096, 7168, 16384])
def test_next_norm_and_codes_have_the_separate_calls_bits(cols, rt, ht):
    g = gen(7 * cols)
    rows = 9
    y, res = rows_of(g, rows, cols, F32), rows_of(g, rows, cols, rt, 8)
    w1, w2 = (1 + 0.2 * torch.randn(cols, generator=g, device=DEV) for _ in range(2))
    N, X = m.Norm(cols, post_w=w1, residual_scale=0.5), m.Norm(cols, pre_w=w2, eps=1e-5)
    out = m.moe_norm_post(N, y, res)
    h = m.moe_norm_pre(X, out, h_dtype=ht)
    out2, h2 = m.moe_norm_post(N, y, res, next_norm=X, h_dtype=ht)
    assert torch.equal(out, out2) and torch.equal(h, h2)
    out3, h3, q, qs = m.moe_norm_post(N, y, res, next_norm=X, h_dtype=ht, quant="block")
    q1, s1 = m.moe_quant_act_q8(h.float())
    assert torch.equal(h3, h) and torch.equal(q, q1) and torch.equal(qs, s1)
    _, h4, q, qs = m.moe_norm_post(N, y, res, next_norm=X, h_dtype=ht, quant="row")
    q1, s1 = m.moe_quant_row_q8(h)
    assert torch.equal(h4, h) and torch.equal(q, q1) and torch.equal(qs, s1)
    # codes alone, of the f32 rows
    none, q, qs = m.moe_norm_pre(X, out, h=False, quant="row")
    q1, s1 = m.moe_quant_row_q8(m.moe_norm_pre(X, out, h_dtype=F32))
    assert none is None and torch.equal(q, q1) and torch.equal(qs, s1)


@pytest.mark.parametrize("cols", [1, 13, 100, 2047])
def test_odd_rows_row_codes(cols):
    g = gen(cols)
    x = rows_of(g, 5, cols, F32, 3)
    h, q, qs = m.moe_norm_pre(m.Norm(cols), x, quant="row")
    q1, s1 = m.moe_quant_row_q8(h)
    assert torch.equal(q, q1) and torch.equal(qs, s1)


@pytest.mark.parametrize("cols", [100, 4096, 8192])
def test_a_row_does_not_depend_on_its_call(cols):
    """Alone, among others, strided, misaligned: the same bits."""
    g = gen(cols + 1)
    x, res = rows_of(g, 33, cols, BF16), rows_of(g, 33, cols, F32)
    w = 1 + 0.2 * torch.randn(cols, generator=g, device=DEV)
    N, X = m.Norm(cols, post_w=w), m.Norm(cols, pre_w=w)
    out, h = m.moe_norm_post(N, x, res, next_norm=X)
    for r in (0, 17, 32):
        o1, h1 = m.moe_norm_post(N, x[r:r + 1], res[r:r + 1], next_norm=X)
        assert torch.equal(o1[0], out[r]) and torch.equal(h1[0], h[r])
    odd = torch.zeros(33 * (cols + 3) + 1, dtype=BF16, device=DEV)[1:].view(33, cols + 3)
    odd[:, :cols] = x
    o2, h2 = m.moe_norm_post(N, odd[:, :cols], res, next_norm=X)
    assert torch.equal(o2, out) and torch.equal(h2, h)


def test_in_place_and_untouched_surroundings():
    g = gen(3)
    for cols, pad in ((4096, 8), (1001, 2)):
        y, res = rows_of(g, 6, cols, F32), rows_of(g, 6, cols, F32, pad)
        N = m.Norm(cols, residual_scale=0.5)
        want = m.moe_norm_post(N, y, res)
        whole = torch.full((8, cols + pad), 9.0, device=DEV)
        inner = whole[1:7, :cols]
        inner.copy_(res)
        got = m.moe_norm_post(N, y, inner, out=inner)
        assert torch.equal(got, want)
        assert (whole[0] == 9).all() and (whole[7] == 9).all() and (whole[:, cols:] == 9).all()
        y2 = y.clone()
        assert torch.equal(m.moe_norm_post(N, y2, res, out=y2), want)
        x2 = y.clone()
        assert torch.equal(m.moe_norm_pre(N, x2, h=x2), m.moe_norm_pre(N, y))
    q = torch.full((6, 1024), 5, dtype=torch.int8, device=DEV)
    m.moe_norm_pre(m.Norm(1001), rows_of(g, 6, 1001, F32), quant="row", q=q[:, :1001])
    assert (q[:, 1001:] == 5).all()


def test_zero_huge_tiny_and_non_finite_rows():
    cols = 4096
    g = gen(4)
    x = torch.randn(6, cols, generator=g, device=DEV)
    x[0] = 0
    x[1] *= 2.0**50
    x[2] *= 1e-30
    x[3, 5] = float("inf")
    x[4, 7] = float("nan")
    N = m.Norm(cols, eps=1e-6)
    h = m.moe_norm_pre(N, x)
    assert (h[0] == 0).all()
    want = ref.rms(ref.f64(x[[1, 2, 5]]), None, float(np.float32(1e-6)))
    # the tiny row's squares underflow under eps: the root is eps's either way
    close(h[[1, 2, 5]], want, np.abs(want), 40, F32)
    bad = h[3]
    assert torch.isnan(bad[5]) and (bad[torch.arange(cols, device=DEV) != 5] == 0).all()
    assert torch.isnan(h[4]).all()
    hq, q, qs = m.moe_norm_pre(N, x[:1], quant="row")
    assert (q == 0).all() and (qs == 0).all()
    assert torch.equal(m.moe_norm_pre(N, x[5:6]), h[5:6])


def test_zero_rows():
    x = torch.empty((0, 64), device=DEV)
    assert m.moe_norm_pre(m.Norm(64), x).shape == (0, 64)
    assert m.moe_norm_post(m.Norm(64), x, x).shape == (0, 64)
    assert m.moe_quant_row_q8(x)[0].shape == (0, 64)


def test_refusals():
    x = torch.zeros((4, 64), device=DEV)
    N = m.Norm(64)
    with pytest.raises(ValueError):
        m.moe_norm_pre(m.Norm(32), x)
    with pytest.raises(ValueError):
        m.moe_norm_pre(N, x.t().contiguous().t())
    with pytest.raises(ValueError):
        m.moe_norm_pre(N, x, quant="column")
    with pytest.raises(ValueError):
        m.moe_norm_post(N, x, x[:3])
    with pytest.raises(ValueError):
        m.moe_norm_post(N, x, x, gate=torch.zeros(3, device=DEV))
    with pytest.raises(TypeError):
        m.moe_norm_post(N, x, x, out=torch.empty_like(x, dtype=BF16))
    with pytest.raises(ValueError):
        m.moe_norm_post(N, x, x, quant="row")
    with pytest.raises(m.MoeError):
        m.moe_norm_pre(m.Norm(16385), torch.zeros((1, 16385), device=DEV))
    with pytest.raises(m.MoeError):
        m.moe_norm_pre(m.Norm(40), torch.zeros((2, 40), device=DEV), quant="block")
    with pytest.raises(m.MoeError):
        m.moe_norm_pre(m.Norm(64, eps=0.0), x)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 8, 0), (5, 100, 0), (2, 4096, 8),
                                           (4, 14336, 0), (3, 20001, 1), (300, 65, 0)])
def test_quant_rows_bit_exact(rows, cols, pad, dtype):
    g = gen(rows * cols)
    x = rows_of(g, rows, cols, dtype, pad, 2.0)
    if rows > 2:
        x[1] = 0
        x[2, -1] = 40.0
    buf = torch.full((rows, (cols + 31) // 16 * 16), 3, dtype=torch.int8, device=DEV)
    q, s = m.moe_quant_row_q8(x, q=buf[:, :cols])
    qr, sr = ref.quant_rows(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)
    assert (buf[:, cols:] == 3).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quant_rows_at_midpoints_and_extreme_scales(dtype):
    """Values on and one step beside every midpoint between codes, and rows whose
    scale is subnormal, tiny, huge or infinite in its reciprocal."""
    half = torch.arange(-126, 127, dtype=torch.float64) + 0.5
    row = torch.cat([half, torch.tensor([127.0])]).float()
    up, down = (torch.nextafter(row, torch.tensor(s)) for s in (np.inf, -np.inf))
    up[-1] = down[-1] = 127.0
    x = torch.stack([row, up, down]).to(DEV)
    rows = [x * 2.0**p for p in (0, -3, 40, -60, -99, -101, -130, -142, -148, 90, 99, 101, 120)]
    rows += [x * f for f in (1.1, 0.3, 7.7, 3e-20)]
    x = torch.cat(rows).to(dtype)
    q, s = m.moe_quant_row_q8(x)
    qr, sr = ref.quant_rows(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)
