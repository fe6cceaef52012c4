"""GPU tests of drafted chains that are deeper than their window: with masks for the window they see what decoding the same
tokens one by one sees (extend_case.py has the references and bounds)."""
import pytest
import torch

from extend_case import BF, E4, ExtendCase
from mxfp4_expert_ffn_router_gb300 import decoder

pytestmark = pytest.mark.gpu


# (few rows a head, and tiles)
@pytest.mark.parametrize("Hq,heads", [(2, 2), (64, 8)])
@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("window,sinks", [(1, 0), (9, 3), (30, 1), (40, 300)])
def test_a_chain_deeper_than_its_window(window, sinks, fmt, Hq, heads):
    plan = [(200, 60), (0, 33), (2, 70), (130, 5), (0, 0)]
    c = ExtendCase(plan, Hq, heads, 64, 32, fmt, seed=window)
    masks, offsets, depths = decoder.tree_masks([list(range(-1, m - 1)) for _, m in plan], window=window, sinks=sinks,
                                                lens=[n for n, _ in plan])
    assert offsets.tolist() == c.offsets.tolist() and depths == [i for _, m in plan for i in range(m)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(*c.run(masks, window=window, sinks=sinks, dev_status=status), window=window, sinks=sinks,
            rows=lambda b, i: Hq == 2 or i % 7 == 0 or i > 55)
    assert status.item() == 0
