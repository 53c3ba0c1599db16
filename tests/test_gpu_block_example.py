"""The whole block of examples/moe_block.py: its rows do not depend on the rows
that share a step (a prefill chunk gives each token what it gets alone, bit for
bit), the operators agree with plain 64-bit forms in their place, and a
captured decode step replays."""
import numpy as np
import pytest
import torch

import block_ref as ref
import synth

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")
from examples.moe_block import Block  # noqa: E402

# (a shape whose decode and prefill kernels share one order of summation; the tiny layer's do not)
SHAPE = synth.Layer(8, 2, 1024, 1024, True)


@pytest.fixture(scope="module")
def block():
    return Block(SHAPE, seed=3)


def rows(n, step=0):
    return torch.from_numpy(synth.activations(3, step, n, SHAPE.d_model)).cuda()


def test_prefill_rows_equal_decoded_rows(block):
    x = rows(70)
    y = block(x)
    assert torch.isfinite(y).all()
    for a, b in ((0, 1), (3, 19), (54, 70)):
        assert torch.equal(block(x[a:b].contiguous()), y[a:b])


def test_operators_in_their_place(block):
    """Each operator against its formula on the inputs that the block gives it."""
    x = rows(33, 1)
    eps = float(np.float32(1e-6))
    h = ref.rms(ref.f64(x), ref.f64(block.pre.tensors[0]), eps)
    _, q, qs = m.moe_norm_pre(block.pre, x, h=False, quant="row")
    # half a code, and what fp32 norms differ by (40 2^-24 of the row's largest, 127 codes)
    assert (np.abs(ref.f64(q) * ref.f64(qs)[:, None] - h)
            <= (0.5 + 127 * 41 * 2.0**-24) * ref.f64(qs)[:, None]).all()
    u = m.moe_linear_q8(block.proj, q, qs)
    w, ws, _ = block.proj.tensors
    assert torch.equal(u.cpu(), ref.linear(q.cpu().numpy(), w.cpu().numpy(), qs.cpu().numpy(),
                                           ws.cpu().numpy(), None, torch.bfloat16))
    x1, h, q, qs = m.moe_norm_post(block.post, u, x, gate=block.gate,
                                   next_norm=block.pre_experts, quant="block")
    b = ref.rms(ref.f64(u), ref.f64(block.post.tensors[1]), eps) * ref.f64(block.gate)
    want = ref.f64(x) + b
    assert (np.abs(ref.f64(x1) - want) <= 48 * 2.0**-24 * (np.abs(ref.f64(x)) + np.abs(b))).all()
    want = ref.rms(ref.f64(x1), ref.f64(block.pre_experts.tensors[0]), eps)
    assert (np.abs(ref.f64(h) - want) <= 40 * 2.0**-24 * np.abs(want)).all()
    ids, wt, counts, offsets, srt = m.moe_route_scored(block.rule,
                                                       m.moe_router_logits(h, block.router))
    for got, want in zip((counts, offsets, srt), ref.group(ids.cpu().numpy(), SHAPE.n_experts)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert torch.allclose(wt.sum(1), torch.full_like(wt[:, 0], 2.5), rtol=1e-6)


def test_captured_decode_step_replays(block):
    x = rows(4, 2)
    want = [block(rows(4, 2 + i)) for i in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x)
    for i in (1, 0, 2, 1, 0):
        x.copy_(rows(4, 2 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(block(x), want[i])   # an eager step between replays
