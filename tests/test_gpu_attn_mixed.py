"""GPU tests of batches in which one sequence has many new tokens and the others few: each goes to the kernels of its own rows."""
import numpy as np
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from extend_case import BF, E4, ExtendCase
from large_case import LargeCase

pytestmark = pytest.mark.gpu


def _plan(prompts):
    plan = [((37 * b) % 150, 1 + (b % 3 == 0)) for b in range(200)]
    for b, p in prompts.items():
        plan[b] = p
    plan[50] = (0, 0)
    return plan


# (a table so wide that the host has to expect long sequences)
@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("Hq,heads,dim", [(8, 4, 128), (8, 2, 64), (3, 3, 256)])
@pytest.mark.parametrize("prompts", [{60: (100, 200)}, {0: (0, 33), 199: (300, 140)}, {}])
def test_a_prompt_among_single_tokens(Hq, heads, dim, prompts, fmt):
    c = ExtendCase(_plan(prompts), Hq, heads, dim, 32, fmt, seed=dim, pad=(1, 2))
    table = np.pad(c.table, ((0, 0), (0, 16384 - c.table.shape[1])), constant_values=-1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    look = lambda b, i: b % 17 == 0 or (b in prompts and (i % 29 == 0 or i > 195))  # noqa: E731
    for window, sinks in ((0, 0), (60, 3)):
        out, lse = c.run(table=table, window=window, sinks=sinks, dev_status=status)
        c.check(out, lse, window=window, sinks=sinks, rows=look)
        again = c.run(table=table, window=window, sinks=sinks, dev_status=status)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    c.check(*c.run(c.trees(4), table=table, dev_status=status), tree=True, rows=look)
    assert status.item() == 0
    offsets = c.offsets.tolist()
    offsets[20] = -1
    out, lse = c.run(offsets=offsets, max_new=200, table=table, dev_status=status)
    assert status.item() == k3.K3MOE_DEV_BOUNDS
    c.check(out, lse, skip=[19, 20], rows=look)


@pytest.mark.parametrize("fmt,heads", [(E4, 32), (BF, 16)])
def test_what_it_costs(fmt, heads):
    """A mixed batch beside its parts: no more than each by itself, and something for the second launches."""
    singles, prompt = [(500, 1)] * 128, [(0, 1900)]
    both, a, b = (LargeCase(p, heads, heads, 128, 64, fmt) for p in (singles + prompt, singles, prompt))
    t, parts = both.us(), a.us(max_new=1) + b.us()
    assert t < 2 * parts + 60, (t, parts)


def test_captured():
    c = LargeCase([(500, 1)] * 128 + [(0, 1900)], 16, 16, 128, 64, BF)
    good = c.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    c.out.fill_(9), c.lse.fill_(9)
    graph.replay()
    assert torch.equal(c.out, good[0]) and torch.equal(c.lse, good[1])


@pytest.mark.parametrize("fmt", [E4, BF])
def test_single_tokens_of_many_heads(fmt):
    """More query heads a key than a sequence of the kernels of few rows has rows: the tiles take single tokens too."""
    plan = [(60 + b % 90, 1) if b % 3 == 0 else (0, 0) for b in range(200)]
    plan[33] = (50, 9)
    c = ExtendCase(plan, 40, 1, 64, 32, fmt, seed=3)
    table = np.pad(c.table, ((0, 0), (0, 60000 - c.table.shape[1])), constant_values=-1)
    c.check(*c.run(table=table), rows=lambda b, i: b % 15 == 0 or b == 33)
