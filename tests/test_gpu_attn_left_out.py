"""GPU tests of values that are not finite where not all rows see them: what a call with one costs beside the same call without
(its other warps wait meanwhile, within a bound), and which rows it reaches."""
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from extend_case import BF, E4
from large_case import LargeCase

pytestmark = pytest.mark.gpu


def _spoil(c, b, p, dims):
    pg, at = c.place(b, p)
    if c.fmt == E4:
        c.cache.v[pg, :, at, dims] = 0x7F  # (a code that is NaN)
    else:
        c.cache.v[pg, :, at, dims] = float("inf")


def _check(c, good, sees, dims, **kw):
    """Rows (of the first sequence) that `sees` names are not finite in those dimensions; all else is as it was."""
    out, lse = c.run(**kw)
    assert c.status.item() == 0 and torch.equal(lse, good[1])
    rows = torch.zeros(c.rows, dtype=torch.bool, device="cuda")
    rows[:len(sees)] = torch.tensor(sees, device="cuda")
    assert torch.equal(out[~rows], good[0][~rows])
    other = [d for d in range(c.dim) if d not in dims]
    assert torch.equal(out[rows][..., other], good[0][rows][..., other])
    assert not torch.isfinite(out[rows][..., dims]).any()


# (128 new tokens in tiles, whole and in parts)
@pytest.mark.parametrize("fmt,dim", [(E4, 128), (BF, 128), (E4, 64), (BF, 256)])
@pytest.mark.parametrize("ctx,m,tree", [(60000, 60, True), (20000, 200, False)])
def test_one_value_in_the_newest_tile(ctx, m, tree, fmt, dim):
    c = LargeCase([(ctx, m), (300, 20)], 64, 8, dim, 64, fmt, tree=tree)
    dims, at = [3, dim - 1], m // 2
    good, before = c.run(), c.us()
    _spoil(c, 0, ctx + at, dims)
    _check(c, good, [i >= at for i in range(m)], dims)
    after = c.us()
    assert after < 4 * before + 200, (before, after)


@pytest.mark.parametrize("fmt", [E4, BF])
def test_in_a_window_and_the_first_tokens(fmt):
    ctx, m, window, sinks = 30000, 150, 5000, 40
    c = LargeCase([(ctx, m), (10, 30)], 64, 8, 128, 64, fmt)
    good, before = c.run(window=window, sinks=sinks), c.us(window=window, sinks=sinks)
    for p in (ctx + 70 - window, 500, ctx - window):  # at the window's edge; before it (where no row sees it)
        _spoil(c, 0, p, [9])
    _check(c, good, [ctx + i - window < ctx + 70 - window for i in range(m)], [9], window=window, sinks=sinks)
    assert c.us(window=window, sinks=sinks) < 4 * before + 200


@pytest.mark.parametrize("fmt", [E4, BF])
def test_beside_a_page_outside_the_cache(fmt):
    """In a tile that all rows see but for a page which the cache has not: all have what is left of it."""
    c = LargeCase([(20000, 60), (300, 20)], 64, 8, 128, 32, fmt, tree=True)
    c.table[0, 101] = c.cache.pages  # (places 3232 .. 3263 of the tile from 3200 on)
    good = c.run()
    assert c.status.item() == k3.K3MOE_DEV_BOUNDS
    for p in (3205, 3300, 3240):
        _spoil(c, 0, p, [p % 5])
    out, _ = c.run()
    dims = [0]  # (3205 and 3300; 3240 lies in the page that is lost, and would be here too)
    assert not torch.isfinite(out[:60][..., dims]).any()
    assert torch.equal(out[:60][..., 1:], good[0][:60][..., 1:]) and torch.equal(out[60:], good[0][60:])


# (few rows a head: a cluster's blocks share an item, or pieces of the line do; 8 and 16 columns)
@pytest.mark.parametrize("fmt,dim", [(E4, 128), (BF, 128), (E4, 64), (BF, 256)])
@pytest.mark.parametrize("plan,Hq,tree", [([(6000, 2)], 32, True), ([(60000, 2), (900, 1)], 64, True), ([(60000, 2), (900, 1)], 32, False)])
def test_one_value_among_few_rows(plan, Hq, tree, fmt, dim):
    c = LargeCase(plan, Hq, 8, dim, 64, fmt, tree=tree)
    dims, (ctx, m) = [3, dim - 1], plan[0]
    good, before = c.run(), c.us()
    _spoil(c, 0, ctx + m - 1, dims)
    _check(c, good, [i == m - 1 for i in range(m)], dims)
    after = c.us()
    assert after < 2.5 * before + 50, (before, after)


def test_a_value_in_the_context_among_few_rows():
    """bf16: left out wherever it lies, and added for all."""
    c = LargeCase([(6000, 2), (50, 3)], 16, 8, 128, 64, BF, tree=True)
    good = c.run()
    for p in (0, 17, 4095, 5999):
        _spoil(c, 0, p, [p % 7])
    _check(c, good, [True, True], sorted({p % 7 for p in (0, 17, 4095, 5999)}))
