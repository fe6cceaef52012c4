"""GPU tests of rows of no sequence in the decoder layer: what comes of them does not depend on the calls before."""
import pytest
import torch

from extend_case import BF, E4, i32
from mxfp4_expert_ffn_router_gb300 import decoder
from test_gpu_decoder_extend import H, PAGE, Model, _bf

pytestmark = pytest.mark.gpu


def _extend(m, layer, pages, counts, masks=None, graph=False):
    """Appends counts[b] tokens and takes them through the layer: (x', a, counts of the experts' rows)."""
    slots = torch.cat([pages.append([b], n) for b, n in enumerate(counts)] + [i32([-1] * (layer.s.T - sum(counts)))])
    offs = i32([0, *torch.tensor(counts).cumsum(0).tolist()])
    x, a = layer.extend(_bf(30, layer.s.T, H), _bf(31, layer.s.T, H), pages.table, pages.seq_lens, slots, offs, masks=masks)
    return x.clone(), a.clone(), layer.counts.clone()


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("fmt", [E4, BF])
def test_more_padding_than_the_call_before(fmt, tree):
    m, counts = Model(fmt, 0, 0, False), [[20, 12], [5, 2]]
    got = []
    for first in ((0, 1), (1,)):  # the second call after the first, and by itself on a new layer
        pages, layer = decoder.PageTable(2, 60, PAGE, 12), m.layer(32)
        if len(first) == 1:
            pages.append([0], 20), pages.append([1], 12)  # (the cache holds the first call's tokens)
        for i in first:
            masks = None
            if tree:
                masks = torch.zeros(32, 1, dtype=torch.int64, device="cuda")
                rows = decoder.tree_masks([list(range(-1, n - 1)) for n in counts[i]])[0]
                masks[:len(rows)] = rows
            out = _extend(m, layer, pages, counts[i], masks)
        got.append(out)
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_a_captured_call_with_other_offsets():
    m = Model(E4, 0, 0, False)
    pages, layer = decoder.PageTable(2, 60, PAGE, 12), m.layer(32)
    slots, offs = torch.cat([pages.append([0], 20), pages.append([1], 12)]), i32([0, 20, 32])
    x = _bf(30, 32, H)
    layer.extend(x, None, pages.table, pages.seq_lens, slots, offs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.extend(x, None, pages.table, pages.seq_lens, slots, offs)
    graph.replay()
    pages.truncate(0, 15), pages.truncate(1, 12)  # five tokens of one sequence are left, and 27 rows of none
    offs.copy_(i32([0, 5, 5])), slots[5:].fill_(-1)
    graph.replay()
    alone = m.layer(32)
    want = alone.extend(x, None, pages.table, pages.seq_lens, slots, offs)
    assert torch.equal(layer.out, want[0]) and torch.equal(layer.a2, want[1]) and torch.equal(layer.counts, alone.counts)
    assert (layer.att[5:] == 0).all() and layer.status.item() == 0
