"""CPU tests of what drafted tokens need on the host: forgetting tokens, positions, and a tree's masks."""
import pytest
import torch

from mxfp4_expert_ffn_router_gb300.decoder import PageTable, tree_masks

PAGE = 16


def _table(lens, pages=20):
    p = PageTable(len(lens), pages, PAGE, 8, device="cpu")
    for b, n in enumerate(lens):
        if n:
            p.append([b], n)
    return p


@pytest.mark.parametrize("lens,b,count,left", [([40, 5], 0, 0, 3), ([40, 5], 0, 7, 3), ([40, 5], 0, 8, 2), ([40, 5], 0, 40, 0),
                                               ([40, 5], 1, 5, 0), ([32], 0, 1, 2), ([33], 0, 1, 2)])
def test_truncate(lens, b, count, left):
    p = _table(lens)
    pages = list(p.owned[b])
    p.truncate(b, count)
    assert p.lens[b] == lens[b] - count and p.owned[b] == pages[:left]
    assert sorted(p.free + [x for o in p.owned for x in o]) == list(range(20))
    assert p.seq_lens.tolist()[b] == lens[b] - count and p.table[b].tolist() == pages[:left] + [-1] * (8 - left)
    again = p.append([b], count)  # the same pages in the same order
    assert p.owned[b] == pages and len(again) == count


@pytest.mark.parametrize("count", [-1, 6])
def test_truncate_refuses(count):
    p = _table([40, 5])
    with pytest.raises(ValueError):
        p.truncate(1, count)
    assert p.lens == [40, 5]


def test_positions():
    p = _table([40, 5])
    assert p.positions_of([0, 1]).tolist() == [39, 4]
    assert p.positions_of([1, 0], 3).tolist() == [2, 3, 4, 37, 38, 39]


def test_tree_masks():
    masks, offsets, depths = tree_masks([[-1, 0, 0, 2], [], [-1, -1, 1]], device="cpu")
    assert masks.tolist() == [[1], [3], [5], [13], [1], [2], [6]]
    assert offsets.tolist() == [0, 4, 4, 7] and depths == [0, 1, 1, 2, 0, 0, 1]
    assert masks.dtype == torch.int64 and offsets.dtype == torch.int32
    chain = list(range(-1, 69))
    masks, _, depths = tree_masks([chain], device="cpu")
    assert masks.shape == (70, 2) and masks[63].tolist() == [-1, 0] and masks[69].tolist() == [-1, 63] and depths == list(range(70))
    masks, offsets, depths = tree_masks([[], []], device="cpu")
    assert masks.shape == (0, 1) and offsets.tolist() == [0, 0, 0] and depths == []


@pytest.mark.parametrize("tree", [[0], [-1, 1], [-1, 2, 0], [-2]])
def test_tree_masks_refuse(tree):
    with pytest.raises(ValueError):
        tree_masks([tree], device="cpu")
