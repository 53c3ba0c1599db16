"""The row quantiser at the longest rows that its argument can name."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

m = pytest.importorskip("mxfp4_routed_expert_e2m1_amd")
DEV = "cuda"


@pytest.mark.parametrize("cols", [2**31 - 1, 2**31 - 8])
def test_the_longest_rows(cols):
    """Every code of a row of 2^31 elements, whose largest one is its last; what lies past the
    row is left alone."""
    n = 1 << 20
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    part = torch.randn(n, generator=g, device=DEV).to(torch.bfloat16)
    x = torch.empty(2**31, dtype=torch.bfloat16, device=DEV)
    x.view(-1, n).copy_(part)
    x[cols - 1] = 9.0
    x[cols:] = 100.0
    q = torch.full((2**31,), 7, dtype=torch.int8, device=DEV)
    _, s = m.moe_quant_row_q8(x[:cols].view(1, cols), q=q[:cols].view(1, cols))
    _, d = ref.quant_rows([[9.0]])
    assert s.item() == d[0]
    # the codes of the repeated part under the row's scale
    want, _ = ref.quant_rows(torch.cat([part.float().cpu(), torch.tensor([9.0])])[None].numpy())
    want = torch.from_numpy(want[0, :n]).to(DEV)
    assert (q[cols:] == 7).all() and q[cols - 1] == 127
    q[cols - 1:] = want[(cols - 1) % n:]
    for i in range(0, 2**31, 1 << 28):
        assert (q[i:i + (1 << 28)].view(-1, n) == want).all(), f"codes from {i} on"
