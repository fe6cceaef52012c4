"""GPU tests of few new tokens for each of more sequences than a block looks through for its item."""
import pytest
import torch

from extend_case import BF, E4, ExtendCase
from large_case import LargeCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("Hq,heads,dim", [(64, 8, 128), (16, 4, 64)])
def test_a_batch_of_one_more_costs_no_more(Hq, heads, dim, tree):
    """256 sequences and 257, max_new left at all rows."""
    few, many = (LargeCase([(500, 2)] * n, Hq, heads, dim, 64, E4, tree=tree) for n in (256, 257))
    a, b = few.us(), many.us()
    assert b < 1.7 * a + 10, (a, b)


# (lengths that one warp, a block, or the line takes)
@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("Hq,heads,ctx", [(16, 1, 40), (8, 1, 300), (4, 2, 60), (16, 1, 1500)])
def test_long_batches(Hq, heads, ctx, tree, fmt):
    plan = [(ctx * (b % 7) // 7, (2, 0, 1, 3, 1)[b % 5]) for b in range(300)]
    plan = [(n if m else 0, m) for n, m in plan]
    c = ExtendCase(plan, Hq, heads, 64, 32, fmt, seed=ctx, pad=(1, 3))
    masks = c.trees(1) if tree else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    look = lambda b, i: b % 11 == 0 or b in (255, 256, 257, 299)  # noqa: E731
    c.check(*c.run(masks, dev_status=status), tree=tree, rows=look)
    c.check(*c.run(masks, window=33, sinks=3, dev_status=status), tree=tree, window=33, sinks=3, rows=look)
    assert status.item() == 0


def test_offsets_out_of_range_in_a_long_batch():
    """Sequences whose offsets are not followed leave their rows as they were; the others' are right."""
    import mxfp4_expert_ffn_router_gb300 as k3
    c = ExtendCase([(20, 2)] * 300, 16, 1, 64, 32, E4, seed=1)
    offsets = c.offsets.tolist()
    offsets[100], offsets[201] = -3, c.rows + 7
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(offsets=offsets, max_new=400, dev_status=status)
    assert status.item() == k3.K3MOE_DEV_BOUNDS
    c.check(out, lse, skip=[99, 100, 200, 201], rows=lambda b, i: b % 9 == 0 or 97 < b < 104)
