"""int8 linear layer: the sum is exact and every later step one rounded fp32
operation, so every output is compared bit for bit."""
import numpy as np
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def codes(rng, rows, cols, pad, lo=-128):
    """int8 view with random bytes between its rows, and the codes alone."""
    ld = (cols + 15) // 16 * 16 + pad
    buf = rng.integers(lo, 128, (rows, ld), dtype=np.int8)
    return torch.from_numpy(buf).to(DEV)[:, :cols], buf[:, :cols]


def check(rows, n, k, dtype=F32, bias=False, pad_q=0, pad_w=0, pad_y=0, seed=0):
    rng = np.random.default_rng([rows, n, k, seed])
    q, qn = codes(rng, rows, k, pad_q)
    w, wn = codes(rng, n, k, pad_w)
    f = lambda c: rng.uniform(0.5, 2.0, c).astype(np.float32) * 2.0**-10  # noqa: E731
    qs, ws = f(rows), f(n)
    b = rng.standard_normal(n).astype(np.float32) if bias else None
    dev = lambda v: None if v is None else torch.from_numpy(v).to(DEV)  # noqa: E731
    lay = m.Linear(w, dev(ws), dev(b))
    whole = torch.full((rows + 1, n + pad_y), 9.0, dtype=dtype, device=DEV)
    y = whole[:rows, :n]
    got = m.moe_linear_q8(lay, q, dev(qs), y=y)
    want = ref.linear(qn, wn, qs, ws, b, dtype)
    assert torch.equal(got.cpu(), want), f"{rows} x {n} x {k}"
    assert (whole[rows] == 9).all() and (whole[:, n:] == 9).all()
    return lay, q, dev(qs), got


ROWS = [1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 257]


@pytest.mark.parametrize("rows", ROWS)
def test_rows(rows):
    for i, (n, k) in enumerate([(96, 256), (130, 1040), (513, 127)]):
        check(rows, n, k, (F32, BF16)[i % 2], bias=i == 1, pad_q=16 * (i % 2), pad_w=16 * i,
              pad_y=i)


@pytest.mark.parametrize("k", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 192,
                               255, 256, 257, 1000, 2050, 4096])
@pytest.mark.parametrize("rows", [1, 7, 40, 130])
def test_row_lengths(rows, k):
    check(rows, 70, k, F32)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 256, 300])
@pytest.mark.parametrize("rows", [1, 16, 50, 300])
def test_channels(rows, n):
    check(rows, n, 320, BF16, bias=n % 2 == 1)


@pytest.mark.parametrize("rows,n,k", [(1, 14336, 4096), (16, 4096, 14336), (33, 4001, 2050),
                                      (100, 2048, 4096), (512, 4096, 2048), (300, 1000, 14336),
                                      (4096, 512, 256), (1000, 2049, 513), (2048, 2304, 640)])
def test_large(rows, n, k):
    check(rows, n, k, BF16 if rows % 2 else F32)


@pytest.mark.parametrize("rows,n,k", [(4096, 14336, 200), (4000, 14300, 321), (2048, 4096, 1000),
                                      (2000, 4001, 130), (1000, 4096, 600), (1500, 3000, 2050)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tiles_of_large_calls(rows, n, k, dtype):
    """The larger tiles, whole and ragged; the sums by a 64-bit product on the GPU (exact: below
    2^53), the later steps in fp32 one at a time."""
    rng = np.random.default_rng([rows, n, k])
    (q, _), (w, _) = codes(rng, rows, k, 16), codes(rng, n, k, 0)
    g = torch.Generator(device=DEV)
    g.manual_seed(k)
    qs, ws = (torch.rand(c, generator=g, device=DEV) + 0.5 for c in (rows, n))
    b = torch.randn(n, generator=g, device=DEV)
    y = m.moe_linear_q8(m.Linear(w, ws, b), q, qs, dtype=dtype)
    want = (q.double() @ w.double().t().contiguous()).round().to(torch.int32).float()
    want = ((want * qs[:, None]) * ws[None, :] + b[None, :]).to(dtype)
    assert torch.equal(y, want)


def test_largest_sums():
    """d_in 65536 of the most negative codes: the sum is 2^30."""
    k = 65536
    for rows in (1, 40):
        q = torch.full((rows, k), -128, dtype=torch.int8, device=DEV)
        w = torch.full((33, k), -128, dtype=torch.int8, device=DEV)
        one = torch.ones(max(rows, 33), device=DEV)
        y = m.moe_linear_q8(m.Linear(w, one[:33]), q, one[:rows], dtype=F32)
        assert (y == 2.0**30).all()


def test_past_four_gigabytes():
    """Weight rows whose byte offsets pass 2^31 and 2^32, token rows as well."""
    k, ld = 256, 65536 * 4
    n = 17000 # 4.4e9 bytes of weight rows, ld apart
    w = torch.empty((n, ld), dtype=torch.int8, device=DEV)[:, :k]
    rng = np.random.default_rng(3)
    wn = rng.integers(-128, 128, (n, k), dtype=np.int8)
    w.copy_(torch.from_numpy(wn))
    one = np.ones(n, dtype=np.float32)
    ones = torch.from_numpy(one).to(DEV)
    for rows in (1, 20, 300):
        qn = rng.integers(-128, 128, (rows, k), dtype=np.int8)
        y = m.moe_linear_q8(m.Linear(w, ones), torch.from_numpy(qn).to(DEV), ones[:rows],
                            dtype=F32)
        assert torch.equal(y.cpu(), ref.linear(qn, wn, one[:rows], one))
    few = w[:40]
    y = m.moe_linear_q8(m.Linear(few.contiguous(), ones[:40]), w, ones, dtype=F32)
    assert torch.equal(y.cpu(), ref.linear(wn, wn[:40], one, one[:40]))


def test_a_row_does_not_depend_on_its_call():
    lay, q, qs, y = check(300, 600, 1000, BF16, bias=True)
    for a, b in ((0, 1), (5, 21), (100, 164), (299, 300)):
        assert torch.equal(m.moe_linear_q8(lay, q[a:b], qs[a:b]), y[a:b])


def test_quantised_on_the_way():
    """Weights and activations through moe_quant_row_q8."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for rows, n, k, dt in ((1, 100, 300, F32), (40, 64, 128, BF16), (3, 257, 2049, BF16)):
        x = torch.randn(rows, k, generator=g, device=DEV).to(dt)
        w = torch.randn(n, k, generator=g, device=DEV)
        lay = m.Linear(*m.moe_quant_row_q8(w))
        y = m.moe_linear_q8(lay, *m.moe_quant_row_q8(x), dtype=F32)
        (qn, qs), (wn, ws) = ref.quant_rows(x.float().cpu().numpy()), ref.quant_rows(w.cpu().numpy())
        assert torch.equal(y.cpu(), ref.linear(qn, wn, qs, ws))


def test_own_stream_graph_and_reused_workspace():
    """Calls on a side stream, and replays of a captured one, against eager
    results; the workspace holds garbage before each."""
    side = torch.cuda.Stream()
    for rows, n, k in ((1, 4096, 4096), (48, 2048, 4096), (200, 512, 8192)):
        lay, q, qs, y = check(rows, n, k, BF16)
        need = m.moe_linear_q8_workspace_bytes(lay, rows)
        ws = torch.randint(-100, 100, (max(need, 16),), device=DEV).to(torch.uint8)
        out = torch.empty_like(y)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m.moe_linear_q8(lay, q, qs, y=out, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(out, y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.moe_linear_q8(lay, q, qs, y=out, ws=ws)
        for i in range(4):
            out.zero_()
            ws.fill_(i + 1)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, y)


def test_zero_rows():
    lay = m.Linear(*m.moe_quant_row_q8(torch.ones((8, 16), device=DEV)))
    q = torch.empty((0, 16), dtype=torch.int8, device=DEV)
    assert m.moe_linear_q8(lay, q, torch.empty(0, device=DEV)).shape == (0, 8)


def test_refusals():
    w = torch.zeros((8, 32), dtype=torch.int8, device=DEV)
    one = torch.ones(8, device=DEV)
    lay = m.Linear(w, one)
    with pytest.raises(ValueError):
        m.moe_linear_q8(lay, torch.zeros((2, 16), dtype=torch.int8, device=DEV), one[:2])
    with pytest.raises(ValueError):
        m.moe_linear_q8(lay, w, one[:3])
    with pytest.raises(TypeError):
        m.moe_linear_q8(lay, w.float(), one)
    with pytest.raises(m.MoeError):   # rows 33 bytes apart
        m.moe_linear_q8(lay, torch.zeros((4, 33), dtype=torch.int8, device=DEV)[:, :32], one[:4])
    with pytest.raises(ValueError):
        m.Linear(w, one[:7])
