"""CPU tests of drafted trees' masks beside a window and first tokens: with the call's rule (drafted tokens by their masks, cached
ones by the window from the position that the number of visible drafted ones gives) a token sees what it would see if its
path were decoded token by token."""
import random

import pytest

from mxfp4_expert_ffn_router_gb300.decoder import tree_masks


def _tree(kind, n, seed):
    rng = random.Random(seed)
    return [i - 1 if kind == "chain" else rng.randrange(max(-1, i - 4), i) for i in range(n)]


def _bits(words):
    x = sum((w % 2 ** 64) << 64 * i for i, w in enumerate(words))
    return {j for j in range(64 * len(words)) if x >> j & 1}


@pytest.mark.parametrize("kind", ["chain", "tree"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (3, 2), (5, 30), (17, 4), (64, 1), (200, 8)])
def test_as_decoded(kind, window, sinks):
    lens = [0, 3, 29, 100]
    trees = [_tree(kind, n, n) for n in (70, 20, 65, 9)]
    masks, offsets, depths = tree_masks(trees, device="cpu", window=window, sinks=sinks, lens=lens)
    for b, (ctx, tree) in enumerate(zip(lens, trees)):
        for i in range(len(tree)):
            row = int(offsets[b]) + i
            path, j = [], i
            while j >= 0:
                path.insert(0, j)
                j = tree[j]
            assert depths[row] == len(path) - 1
            p = ctx + depths[row]  # decoded: place c <= p is seen if c > p - window or c < sinks
            want = {c for c in range(p + 1) if c > p - window or c < sinks}
            named = _bits(masks[row].tolist())
            # the call: the context by the window from n - m + max(0, named - 1), drafted tokens by the mask
            q = ctx + max(0, len(named) - 1)
            got = {c for c in range(ctx) if c > q - window or c < sinks} | {ctx + path.index(j) for j in named}
            assert got == want, (b, i)


def test_without_a_window_they_are_as_before():
    trees = [_tree("tree", 70, 1), [], _tree("chain", 5, 2)]
    a, b = tree_masks(trees, device="cpu"), tree_masks(trees, device="cpu", window=71)
    assert a[0].tolist() == b[0].tolist() and a[1].tolist() == b[1].tolist() and a[2] == b[2]
    assert tree_masks(trees, device="cpu", sinks=4)[0].tolist() == a[0].tolist()  # (sinks mean something beside a window)


@pytest.mark.parametrize("kw", [dict(window=-1), dict(sinks=-1), dict(window=4, sinks=2), dict(window=4, sinks=2, lens=[1, 2])])
def test_refused(kw):
    with pytest.raises(ValueError):
        tree_masks([[-1, 0]], device="cpu", **kw)
