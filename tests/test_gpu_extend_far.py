"""GPU tests of the calls of several new tokens at offsets past 32 bits, of two calls at once, and after others that leave
large queries in shared memory: the same results, bit for bit, as near the start of a small cache, or alone."""
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from extend_case import BF, E4, ExtendCase, dev, i32

pytestmark = pytest.mark.gpu

TILES = [(700, 61), (0, 55), (256, 70)]
FEW = [(700, 3), (0, 2), (256, 1)]
ONE = [(700, 1), (0, 1), (256, 1)]


def _far(c):
    """The case's cache as the last pages of one whose vectors pass 2^32 bytes, and the table that names them."""
    small = c.cache
    per_page = small.k[0].numel() * small.k.element_size()
    pages = (2 ** 32 + 2 ** 20) // per_page + small.pages + 1
    big = k3.KVCache.empty(pages, small.heads, small.page_size, small.dim, small.format)
    for name in ("k", "v", "k_scales", "v_scales"):
        if getattr(small, name) is not None:
            getattr(big, name)[pages - small.pages:].copy_(getattr(small, name))
    assert (pages - small.pages) * per_page > 2 ** 32
    return big, pages - small.pages


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("plan,tree", [(TILES, False), (TILES, True), (FEW, False), (FEW, True), (ONE, False)])
def test_pages_past_32_bits(plan, tree, fmt):
    c = ExtendCase(plan, 27, 9, 128, 64, fmt, seed=7)
    masks = c.trees(2) if tree else None
    most = None if tree else max(m for _, m in plan)
    want = c.run(masks, window=300, sinks=5, max_new=most)
    c.cache, first = _far(c)
    got = c.run(masks, window=300, sinks=5, max_new=most, table=c.table + (c.table >= 0) * first)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("fmt", [E4, BF])
def test_appending_past_32_bits(fmt):
    c = ExtendCase(FEW, 18, 9, 128, 64, fmt, seed=8)
    n = len(c.slots)
    k, v = (dev(c.rng.integers(0x3F00, 0x4080, (n, 9, 128)).astype("uint16")) for _ in range(2))
    pos, rotation = i32(range(n)), k3.Rotation(64)
    big, first = _far(c)
    out = []
    for cache, slots in ((c.cache, c.slots), (big, c.slots + first * 64)):
        k3.k3moe_kv_append(cache, k, v, slots, pos, rotation)
        kv = [torch.empty_like(k) for _ in range(2)]
        k3.k3moe_kv_read(cache, slots, *kv)
        out.append(kv)
    assert all(torch.equal(x, y) for x, y in zip(*out))


@pytest.mark.parametrize("first,second", [(TILES, FEW), (TILES, TILES), (FEW, ONE)])
def test_two_calls_at_once(first, second):
    cases = [ExtendCase(first, 27, 9, 128, 64, E4, seed=1), ExtendCase(second, 27, 9, 128, 64, BF, seed=2)]
    want = [c.run(window=200, sinks=3, max_new=max(m for _, m in c.plan)) for c in cases]
    calls = [(c, dev(c.q_bits), c.args(), c.workspace(), [c.outputs() for _ in range(8)], torch.cuda.Stream()) for c in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for c, q, args, ws, outs, st in calls:
            k3.k3moe_attn_extend(c.cache, q, *args, outs[i][0], lse=outs[i][1], window=200, sinks=3,
                                 max_new=max(m for _, m in c.plan), ws=ws, stream=st)
    torch.cuda.synchronize()
    for (c, _, _, _, outs, _), w in zip(calls, want):
        assert all(torch.equal(x, y) for o in outs for x, y in zip(o, w))


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_after_a_call_with_large_queries(dim, fmt):
    # the last warp of an item has rows without a query
    cases = [ExtendCase(TILES, 27, 9, dim, 64, fmt, seed=3)]
    cases += [ExtendCase([(700, 256), (0, 256)], 32, 8, dim, 64, fmt, seed=4, q_scale=s) for s in (1e-3, 300.0)]
    calls = [(c, dev(c.q_bits), c.args(), c.workspace(), [c.outputs() for _ in range(6)]) for c in cases]
    torch.cuda.synchronize()

    def call(i, r):
        c, q, args, ws, outs = calls[i]
        k3.k3moe_attn_extend(c.cache, q, *args, outs[r][0], lse=outs[r][1], window=200, sinks=3, ws=ws)

    for r in range(6):  # after small ones, and after large ones: nothing else runs between, which would use the same memory
        for _ in range(2):
            call(1 if r < 3 else 2, r)
        call(0, r)
    torch.cuda.synchronize()
    runs = calls[0][4]
    assert all(torch.equal(x, y) for r in runs[1:] for x, y in zip(r, runs[0]))
