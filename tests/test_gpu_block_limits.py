"""The operators around the experts at their edges: rows that are not numbers
through the int8 path, more rows than one launch takes, calls on a stream that
is not the current one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# (rows in one wave, in several, in registers past one unit, and read twice)
@pytest.mark.parametrize("cols", [5, 100, 2049, 5000, 16384, 40000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_row_codes_of_rows_that_are_not_numbers(cols, dtype):
    """A NaN anywhere in a row makes its scale NaN, an infinity not finite, so
    the layer that reads the codes does not take the row for zeros; the rows
    beside it keep their bits."""
    x = torch.randn((6, cols), generator=gen(cols), device=DEV).to(dtype)
    q0, s0 = m.moe_quant_row_q8(x)
    bad = x.clone()
    bad[1, cols - 1] = float("nan")
    bad[2, cols // 2] = float("inf")
    bad[3] = float("nan")
    bad[4, 0] = -float("nan")
    q, s = m.moe_quant_row_q8(bad)
    assert torch.isnan(s[[1, 3, 4]]).all() and not torch.isfinite(s[2])
    assert torch.equal(q[[0, 5]], q0[[0, 5]]) and torch.equal(s[[0, 5]], s0[[0, 5]])
    if cols <= 16384:
        _, q, s = m.moe_norm_pre(m.Norm(cols), bad, h=False, quant="row")
        assert torch.isnan(s[1:5]).all() and torch.isfinite(s[[0, 5]]).all()
        w = torch.randn((40, cols), generator=gen(1), device=DEV)
        y = m.moe_linear_q8(m.Linear(*m.moe_quant_row_q8(w)), q, s)
        assert torch.isnan(y[1:5]).all() and torch.isfinite(y[[0, 5]]).all()


def test_more_rows_than_a_launch():
    """Rows from 2^21 on, which go in a launch of their own, have the bits they
    have alone."""
    rows, cols = (1 << 21) + 3, 8
    x = torch.randn((rows, cols), generator=gen(2), device=DEV)
    ends = torch.tensor([0, 1, (1 << 21) - 1, 1 << 21, rows - 1], device=DEV)
    q, s = m.moe_quant_row_q8(x)
    N = m.Norm(cols)
    h = m.moe_norm_pre(N, x)
    out = m.moe_norm_post(N, x, h, gate=s.view(rows, 1))
    some = x[ends].contiguous()
    qe, se = m.moe_quant_row_q8(some)
    he = m.moe_norm_pre(N, some)
    assert torch.equal(q[ends], qe) and torch.equal(s[ends], se)
    assert torch.equal(h[ends], he)
    assert torch.equal(out[ends], m.moe_norm_post(N, some, he, gate=se.view(-1, 1)))


def test_another_stream_keeps_its_buffers():
    """A call on a busy stream has not run when it returns: what it allocated,
    its workspace too, must not be handed to the current stream before then."""
    side = torch.cuda.Stream()
    g = gen(3)
    z = torch.randn((777, 272), generator=g, device=DEV)
    x = torch.randn((48, 14336), generator=g, device=DEV)
    w = torch.randn((1024, 14336), generator=g, device=DEV)
    lay, rule, N = m.Linear(*m.moe_quant_row_q8(w)), m.RouterRule(272, 8), m.Norm(14336)
    q, s = m.moe_quant_row_q8(x)
    want = [*m.moe_route_scored(rule, z), m.moe_linear_q8(lay, q, s), *m.moe_quant_row_q8(x),
            m.moe_norm_pre(N, x), m.moe_norm_post(N, x, x)]
    needs = [m.moe_route_scored_workspace_bytes(rule, 777),
             m.moe_linear_q8_workspace_bytes(lay, 48)]
    assert min(needs) > 0
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000)
    got = [*m.moe_route_scored(rule, z, stream=side), m.moe_linear_q8(lay, q, s, stream=side),
           *m.moe_quant_row_q8(x, stream=side), m.moe_norm_pre(N, x, stream=side),
           m.moe_norm_post(N, x, x, stream=side)]
    taken = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in needs for _ in range(8)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all((t == 255).all() for t in taken)


def test_given_buffers_on_a_given_stream():
    side = torch.cuda.Stream()
    g = gen(4)
    z = torch.randn((777, 160), generator=g, device=DEV)
    x = torch.randn((48, 4096), generator=g, device=DEV)
    w = torch.randn((512, 4096), generator=g, device=DEV)
    lay, rule, N = m.Linear(*m.moe_quant_row_q8(w)), m.RouterRule(160, 6), m.Norm(4096)
    q, s = m.moe_quant_row_q8(x)
    want = [*m.moe_route_scored(rule, z), m.moe_linear_q8(lay, q, s), q, s,
            *m.moe_norm_post(N, x, x, next_norm=N, quant="row")]
    route, y = m.route_outputs(777, 160, 6), torch.empty_like(want[5])
    wr = torch.empty(m.moe_route_scored_workspace_bytes(rule, 777), dtype=torch.uint8, device=DEV)
    wl = torch.empty(max(m.moe_linear_q8_workspace_bytes(lay, 48), 16), dtype=torch.uint8,
                     device=DEV)
    q2, s2, out, h = m.codes_buffer(48, 4096), torch.empty_like(s), *torch.empty((2, 48, 4096),
                                                                                 device=DEV)
    q3, s3 = m.codes_buffer(48, 4096), torch.empty_like(s)
    torch.cuda.synchronize()
    m.moe_route_scored(rule, z, out=route, ws=wr, stream=side)
    m.moe_quant_row_q8(x, q=q2, scales=s2, stream=side)
    m.moe_linear_q8(lay, q2, s2, y=y, ws=wl, stream=side)
    m.moe_norm_post(N, x, x, out=out, next_norm=N, h=h, quant="row", q=q3, qs=s3, stream=side)
    side.synchronize()
    for a, b in zip([*route, y, q2, s2, out, h, q3, s3], want, strict=True):
        assert torch.equal(a, b)
