"""GPU tests of k3moe_attn_extend and k3moe_attn_tree where a sequence has many rows a head, so that the kernels of tiles
take the call: blocks of one item, items shared by blocks, and pieces of a line of items (extend_case.py has the bounds)."""
import numpy as np
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from extend_case import BF, E4, ExtendCase

pytestmark = pytest.mark.gpu

# (places before, new tokens): a block an item; items in parts; a line; a line whose items are cut; rows behind G that is odd
ONE = ([(60, 50), (0, 64), (0, 0), (17, 33)], 64, 8)
PARTS = ([(1900, 40)], 64, 8)
LINE = ([(100, 40), (0, 90), (300, 35), (5, 60), (0, 0), (129, 50), (64, 64)], 48, 8)
CUT = ([(2500, 40), (10, 130), (900, 3), (0, 300)], 64, 8)
ODD = ([(700, 61), (0, 55), (256, 70)], 27, 9)


def _look(b, i):
    return i % 13 == 0 or i in (1, 31, 32, 39)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("dim,page", [(64, 32), (128, 64), (128, 16), (256, 128)])
@pytest.mark.parametrize("shape", [ONE, PARTS, LINE, CUT, ODD])
def test_prompts_and_trees(shape, dim, page, fmt):
    plan, Hq, heads = shape
    c = ExtendCase(plan, Hq, heads, dim, page, fmt, seed=dim + page + len(plan), pad=(2, 3))
    c.check(*c.run(), rows=_look)
    c.check(*c.run(window=150, sinks=5), window=150, sinks=5, rows=_look)
    words = -(-max(m for _, m in plan) // 64)
    c.check(*c.run(c.trees(words)), tree=True, rows=_look)
    c.check(*c.run(c.trees(words, "any"), window=333, sinks=130), tree=True, window=333, sinks=130, rows=_look)


@pytest.mark.parametrize("shape", [PARTS, LINE, CUT])
@pytest.mark.parametrize("stale", ["nan", "inf"])
@pytest.mark.parametrize("fmt,dim", [(E4, 64), (E4, 128), (E4, 256), (BF, 64), (BF, 128), (BF, 256)])
def test_values_that_a_row_does_not_see(shape, fmt, dim, stale):
    """Tokens of the sequence that hold NaN or infinities touch the rows that see them, and those alone."""
    plan, Hq, heads = shape
    c = ExtendCase(plan, Hq, heads, dim, 32, fmt, seed=5, stale=stale)
    at, slots, hidden = 0, c.slots.cpu().numpy(), {}
    for b, (ctx, m) in enumerate(plan):
        hidden[b] = np.zeros(ctx + m, bool)
        if m:
            hidden[b][[ctx + m // 2, ctx + m - 1]] = True
        for p in np.flatnonzero(hidden[b]):
            pg, pl = divmod(int(slots[at + p]), 32)
            if fmt == BF:
                c.cache.v[pg, :, pl, 1::3] = float(stale)
            elif stale == "nan":
                c.cache.v_scales[pg, :, pl] = 255
            else:
                c.cache.v[pg, :, pl, ::5] = 0x7F  # (a code that is NaN)
        at += ctx + m
    for window, sinks, tree in [(0, 0, False), (30, 2, False), (0, 0, True)]:
        masks = c.trees(-(-max(m for _, m in plan) // 64)) if tree else None
        out, lse = c.run(masks, window=window, sinks=sinks)

        def sees_bad(b, i):
            return bool((c.seen(b, i, tree, window, sinks) & hidden[b]).any())

        c.check(out, lse, tree=tree, window=window, sinks=sinks, rows=lambda b, i: not sees_bad(b, i) and _look(b, i))
        finite = torch.isfinite(out.float()).all(-1).all(-1).cpu().numpy()
        for b, (ctx, m) in enumerate(plan):
            for i in range(m):
                assert finite[int(c.offsets[b]) + i] != sees_bad(b, i), (b, i)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("shape", [ONE, PARTS, LINE])
def test_scores_that_grow_and_values_of_every_size(shape, fmt):
    """A row's reference moves where later places score far higher, in either half of a tile and between tiles."""
    plan, Hq, heads = shape

    def kv(rng, n):
        import decoder_ref as ref
        k = rng.standard_normal((n, heads, 128)) * (2.0 ** (np.arange(n) % 97 / 12))[:, None, None]
        v = rng.standard_normal((n, heads, 128)) * 2.0 ** rng.integers(-18, 19, (n, heads, 1))
        return ref.bf16_bits(k), ref.bf16_bits(v)

    c = ExtendCase(plan, Hq, heads, 128, 64, fmt, seed=8, kv=kv, q_scale=0.7)
    c.check(*c.run(), rows=_look)
    c.check(*c.run(window=90, sinks=3, scale=-0.3), window=90, sinks=3, scale=-0.3, rows=_look)


@pytest.mark.parametrize("fmt", [E4, BF])
def test_codes_and_scales_at_their_ends(fmt):
    """Scales of 2^-127 (all zeros) to the largest that bf16 holds, beside ordinary ones."""
    plan, Hq, heads = CUT

    def kv(rng, n):
        import decoder_ref as ref
        v = rng.standard_normal((n, heads, 128))
        v[::7] = 0
        v[3::11] *= 2.0 ** 100
        v[5::11] *= 2.0 ** -100
        k = rng.standard_normal((n, heads, 128))
        k[::9] = 0
        k[4::13] *= 2.0 ** -60
        return ref.bf16_bits(k), ref.bf16_bits(v)

    c = ExtendCase(plan, Hq, heads, 128, 64, fmt, seed=3, kv=kv)
    c.check(*c.run(), rows=_look)


@pytest.mark.parametrize("tree", [False, True])
def test_pages_outside_the_cache(tree):
    plan, Hq, heads = CUT
    c = ExtendCase(plan, Hq, heads, 128, 64, E4, seed=4)
    masks = c.trees(5) if tree else None
    table = c.table.copy()
    table[0, 7], table[0, 39], table[1, 1], table[3, 2] = c.cache.pages, -9, 0x7FFFFFFF, -1
    hidden = {b: np.zeros(ctx + m, bool) for b, (ctx, m) in enumerate(plan)}
    for b, p in ((0, 7), (0, 39), (1, 1), (3, 2)):
        hidden[b][64 * p:64 * p + 64] = True
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(*c.run(masks, table=table, dev_status=status), tree=tree, hidden=hidden, rows=_look)
    assert status.item() == k3.K3MOE_DEV_BOUNDS
    # those before a window are not looked up
    table = c.table.copy()
    table[0, 1:36], status = -1, status.zero_()
    out = c.run(masks, window=170, sinks=20, table=table, dev_status=status)
    c.check(*out, tree=tree, window=170, sinks=20, rows=_look)
    assert status.item() == 0


def test_offsets_out_of_range():
    plan, Hq, heads = LINE
    c = ExtendCase(plan, Hq, heads, 128, 64, BF, seed=1, pad=(0, 4))
    good = c.offsets.tolist()
    for bad, skip in (({0: -1}, [0]), ({7: c.rows + 5}, [6]), ({3: good[2] - 1}, [2, 3])):
        offsets = [bad.get(i, o) for i, o in enumerate(good)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # (a sequence behind one whose offsets descend would span 96 rows: more than max_new)
        out, lse = c.run(offsets=offsets, dev_status=status, max_new=95)
        assert status.item() == k3.K3MOE_DEV_BOUNDS
        c.check(out, lse, skip=skip, rows=_look)
    lens = list(c.lens)
    lens[1], lens[5] = 30, -4  # fewer places than new tokens
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(lens=lens, dev_status=status)
    assert status.item() == k3.K3MOE_DEV_BOUNDS
    c.check(out, lse, rows=lambda b, i: b not in (1, 5) and _look(b, i))
    none = slice(int(c.offsets[1]), int(c.offsets[1]) + 60)
    assert (out[none] == 0).all() and (lse[none] == -np.inf).all()
    none = slice(int(c.offsets[5]), int(c.offsets[6]))
    assert (out[none] == 0).all() and (lse[none] == -np.inf).all()


@pytest.mark.parametrize("shape", [ONE, PARTS, CUT])
def test_captured_twice_over_one_workspace(shape):
    """Two calls of different shapes, captured into two graphs that share a workspace, replayed in turn."""
    plan, Hq, heads = shape
    a = ExtendCase(plan, Hq, heads, 128, 64, E4, seed=2)
    b = ExtendCase([(300, 9), (0, 70)], Hq, heads, 128, 64, BF, seed=3)
    ws = max(a.workspace(), b.workspace(), key=lambda t: t.numel())
    calls = []
    for c in (a, b):
        import extend_case
        q, args, (out, lse) = extend_case.dev(c.q_bits), c.args(), c.outputs()

        def call(c=c, q=q, args=args, out=out, lse=lse):
            k3.k3moe_attn_extend(c.cache, q, *args, out, lse=lse, window=200, sinks=3, ws=ws)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        calls.append((c, graph, out, lse))
    for _ in range(3):
        for c, graph, out, lse in calls:
            out.fill_(9), lse.fill_(9)
            graph.replay()
    for c, graph, out, lse in calls:
        c.check(out, lse, window=200, sinks=3, rows=_look)
