"""GPU tests of k3moe_attn_extend and k3moe_attn_tree against float64 references (extend_case.py)."""
import numpy as np
import pytest
import torch

import decoder_ref as ref
import mxfp4_expert_ffn_router_gb300 as k3
from extend_case import BF, E4, ExtendCase, dev, i32

pytestmark = pytest.mark.gpu

SHORT = [(0, 1), (1, 1), (0, 0), (15, 2), (16, 16), (63, 5), (64, 1), (0, 17), (130, 3), (257, 9), (0, 0)]
LONG = [(1000, 7), (127, 2), (0, 140), (128, 128), (300, 33)]
HEADS = [(8, 8, 128, 64), (8, 1, 128, 16), (12, 4, 64, 32), (10, 2, 256, 64), (16, 1, 64, 128), (9, 1, 128, 1024),
         (3, 3, 256, 16), (40, 1, 128, 32)]


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("Hq,heads,dim,page", HEADS)
def test_prompts(Hq, heads, dim, page, fmt):
    c = ExtendCase(SHORT, Hq, heads, dim, page, fmt, seed=dim + Hq, pad=(3, 5))
    c.check(*c.run())


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("Hq,heads,dim,page", [(8, 2, 128, 64), (4, 4, 64, 16), (5, 1, 256, 32)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (20, 4), (128, 130), (300, 3), (129, 0), (5000, 7)])
def test_window_and_sinks(Hq, heads, dim, page, fmt, window, sinks):
    c = ExtendCase(LONG, Hq, heads, dim, page, fmt, seed=window + dim)
    c.check(*c.run(window=window, sinks=sinks), window=window, sinks=sinks, rows=lambda b, i: i % 5 == 0 or i > 120)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("Hq,heads,dim,page", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 4), (3, 0)])
def test_single_tokens(Hq, heads, dim, page, fmt, window, sinks):
    plan = [(0, 1), (1, 1), (0, 0), (15, 1), (64, 1), (130, 1), (257, 1), (999, 1), (2, 1)]
    c = ExtendCase(plan, Hq, heads, dim, page, fmt, seed=dim + Hq + window, pad=(1, 2))
    c.check(*c.run(window=window, sinks=sinks, max_new=1), window=window, sinks=sinks)
    c.check(*c.run(window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("Hq,heads,dim,page", HEADS)
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_trees(Hq, heads, dim, page, fmt, kind):
    c = ExtendCase([(50, 8), (0, 5), (3, 1), (0, 0), (300, 64), (127, 13), (640, 20)], Hq, heads, dim, page, fmt,
                   seed=dim + Hq, pad=(0, 4))
    m = c.trees(1, kind)
    c.check(*c.run(m), tree=True)


@pytest.mark.parametrize("words,plan", [(1, [(200, 64), (5, 63)]), (2, [(100, 65), (0, 128), (300, 7), (0, 0)]), (3, [(33, 150)]),
                                        (16, [(10, 300), (700, 1)])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (1, 0), (400, 130)])
def test_tree_words_and_windows(words, plan, window, sinks):
    c = ExtendCase(plan, 4, 2, 64, 16, E4, seed=words + window)
    for kind in ("tree", "any"):
        c.check(*c.run(c.trees(words, kind), window=window, sinks=sinks), tree=True, window=window, sinks=sinks,
                rows=lambda b, i: i % 7 == 0 or i > 280)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("plan,Hq,heads,dim,page", [([(5000, 6), (4, 2)], 8, 1, 128, 64), ([(20000, 3)], 4, 2, 64, 128),
                                                    ([(3000, 40)] * 3, 2, 1, 256, 16), ([(700, 2)] * 40, 4, 1, 128, 32),
                                                    ([(0, 600), (9000, 1), (0, 0), (33, 90)], 4, 2, 128, 64)])
def test_long_caches(plan, Hq, heads, dim, page, fmt):
    """Long sequences are split over the GPU and joined."""
    c = ExtendCase(plan, Hq, heads, dim, page, fmt, seed=len(plan))
    look = lambda b, i: b < 4 and (i % 37 == 0 or i < 4)  # noqa: E731
    c.check(*c.run(), rows=look)
    c.check(*c.run(window=2000, sinks=5), window=2000, sinks=5, rows=look)
    m = max(m for _, m in plan)
    if m <= 64:
        c.check(*c.run(c.trees(1)), tree=True, rows=look)


def test_a_chain_is_a_prompt():
    c = ExtendCase([(200, 30), (0, 64), (1000, 1)], 8, 2, 128, 32, E4)
    a, b = c.run(), c.run(c.trees(1, "chain"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("stale", ["nan", "inf"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_that_a_row_does_not_see_do_not_touch_it(fmt, stale, dim):
    """Tokens of the sequence itself that hold NaN or infinities: rows that see them have them, others not."""
    plan, bad = [(150, 40), (0, 200), (300, 20)], {0: [160, 3], 1: [90, 199], 2: [0, 305]}
    c = ExtendCase(plan, 4, 2, dim, 32, fmt, seed=5)
    at, slots = 0, c.slots.cpu().numpy()
    hidden = {}
    for b, (ctx, m) in enumerate(plan):
        hidden[b] = np.zeros(ctx + m, bool)
        hidden[b][bad[b]] = True
        for p in bad[b]:
            pg, pl = divmod(int(slots[at + p]), 32)
            if fmt == BF:
                c.cache.v[pg, :, pl, 1::3] = float(stale)
                c.cache.k[pg, :, pl, 5] = float(stale)
            else:
                c.cache.v_scales[pg, :, pl] = 255
                c.cache.k_scales[pg, :, pl] = 255
        at += ctx + m
    for window, sinks, tree in [(0, 0, False), (30, 2, False), (0, 0, True), (25, 1, True)]:
        masks = c.trees(4, "tree") if tree else None
        out, lse = c.run(masks, window=window, sinks=sinks)

        def sees_bad(b, i):
            return bool((c.seen(b, i, tree, window, sinks) & hidden[b]).any())

        c.check(out, lse, tree=tree, window=window, sinks=sinks, rows=lambda b, i: not sees_bad(b, i))
        for b, (ctx, m) in enumerate(plan):
            for i in range(m):
                if sees_bad(b, i):
                    assert not torch.isfinite(out[int(c.offsets[b]) + i].float()).all(), (b, i)


@pytest.mark.parametrize("stale", ["nan", "inf"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_that_are_not_finite(stale, dim):
    """V alone holds NaN or infinities (K finite): elements of rows that see them are as in 64 bits, the others finite."""
    plan, places = [(150, 40), (0, 200)], [[160, 3], [90, 130]]
    c = ExtendCase(plan, 4, 2, dim, 32, BF, seed=6)
    at, slots = 0, c.slots.cpu().numpy()
    for b, (ctx, m) in enumerate(plan):
        for p in places[b]:
            pg, pl = divmod(int(slots[at + p]), 32)
            c.cache.v[pg, :, pl, 1::3] = float(stale)
            c.v[at + p, :, 1::3] = float(stale)
        at += ctx + m
    out, lse = c.run(window=50, sinks=3)
    got = out.double().cpu().numpy()
    at = 0
    for b, (ctx, m) in enumerate(plan):
        for i in range(m):
            see = c.seen(b, i, False, 50, 3)
            bad = ~np.isfinite(c.v[at:at + ctx + m][see][:, 0]).all(0) if see.any() else np.zeros(dim, bool)
            r = got[int(c.offsets[b]) + i]
            assert np.isfinite(r[:, ~bad]).all(), (b, i)
            assert (np.isnan(r[:, bad]) if stale == "nan" else r[:, bad] == np.inf).all(), (b, i)
        at += ctx + m


@pytest.mark.parametrize("fmt", [E4, BF])
def test_large_and_small_scores(fmt):
    """Scores of thousands (one place takes the whole weight) and values of very different size."""
    for spread, q_scale in ((0, 300.0), (20, 1.0)):
        c = ExtendCase([(400, 30), (0, 64)], 4, 1, 128, 64, fmt, seed=9, spread=spread, q_scale=q_scale)
        c.check(*c.run(), rows=lambda b, i: i % 3 == 0)
        c.check(*c.run(window=100, sinks=4, scale=-0.5), window=100, sinks=4, scale=-0.5, rows=lambda b, i: i % 3 == 0)


@pytest.mark.parametrize("tree", [False, True])
def test_pages_outside_the_cache(tree):
    """Their places count as not seen; what other rows see is unharmed."""
    plan = [(100, 20), (600, 30), (0, 40)]
    c = ExtendCase(plan, 4, 2, 128, 32, E4, seed=4)
    masks = c.trees(1) if tree else None
    table = c.table.copy()
    table[0, 1], table[1, 17], table[2, 1] = c.cache.pages, -5, 0x7FFFFFFF
    hidden = {0: np.zeros(120, bool), 1: np.zeros(630, bool), 2: np.zeros(40, bool)}
    hidden[0][32:64], hidden[1][544:576], hidden[2][32:] = True, True, True
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(*c.run(masks, table=table, dev_status=status), tree=tree, hidden=hidden)
    assert status.item() == k3.K3MOE_DEV_BOUNDS
    status.zero_()
    c.check(*c.run(masks, dev_status=status), tree=tree)
    assert status.item() == 0


def test_pages_before_the_window_are_not_looked_up():
    c = ExtendCase([(1000, 8)], 4, 2, 64, 128, E4, seed=2)
    table = c.table.copy()
    table[0, 1:6] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(*c.run(window=200, sinks=100, table=table, dev_status=status), window=200, sinks=100)
    assert status.item() == 0
    c.check(*c.run(c.trees(1), window=200, sinks=100, table=table, dev_status=status), window=200, sinks=100, tree=True)
    assert status.item() == 0


def test_offsets_and_lengths_out_of_range():
    plan = [(20, 4), (30, 5), (40, 6), (9, 3)]
    c = ExtendCase(plan, 4, 2, 64, 16, BF, seed=1, pad=(0, 3))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for offsets, skip in [([-1, 4, 9, 15, 18], [0]), ([0, 4, 9, 15, 40], [3]), ([0, 4, 9, 3, 18], [2, 3])]:
        status.zero_()
        out, lse = c.run(offsets=offsets, dev_status=status, max_new=6)
        assert status.item() == k3.K3MOE_DEV_BOUNDS
        c.check(out, lse, skip=skip)
    status.zero_()  # more new tokens than max_new
    out, lse = c.run(max_new=5, dev_status=status)
    assert status.item() == k3.K3MOE_DEV_BOUNDS
    c.check(out, lse, skip=[2])
    status.zero_()  # fewer cached tokens than new ones: the rows without a place see nothing
    out, lse = c.run(lens=[24, 2, 46, -7], dev_status=status)
    assert status.item() == k3.K3MOE_DEV_BOUNDS
    c.check(out, lse, rows=lambda b, i: b in (0, 2))
    assert (out[4:7] == 0).all() and (lse[4:7] == -np.inf).all() and torch.isfinite(lse[7:9]).all()
    assert (out[15:18] == 0).all() and (lse[15:18] == -np.inf).all()
    status.zero_()  # longer than the table
    out, lse = c.run(lens=[24, 35, 46, 10 ** 6], dev_status=status, table=c.table)
    assert status.item() == k3.K3MOE_DEV_BOUNDS
    c.check(out, lse, rows=lambda b, i: b < 3)


def test_strides_streams_and_no_lse():
    c = ExtendCase([(70, 9), (0, 20), (500, 3)], 8, 2, 128, 64, E4, seed=3)
    want = c.run()
    wide = torch.full((c.rows, 12, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = dev(c.q_bits)
    got = c.run(q=wide[:, :8])
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    args = c.args()
    out, lse = c.outputs()
    q, ws = dev(c.q_bits), c.workspace()
    torch.cuda.synchronize()
    k3.k3moe_attn_extend(c.cache, q, *args, out, lse=lse, ws=ws, stream=st)
    st.synchronize()
    assert torch.equal(want[0], out) and torch.equal(want[1], lse)
    out, lse = c.run(lse=False)
    assert torch.equal(want[0], out) and (lse == 9).all()


@pytest.mark.parametrize("tree", [False, True])
def test_captured_calls_follow_lengths_and_offsets(tree):
    c = ExtendCase([(70, 9), (300, 20), (500, 3)], 8, 2, 128, 64, E4, seed=3)
    d = ExtendCase([(71, 1), (0, 12), (600, 19)], 8, 2, 128, 64, E4, seed=8)
    offs, table, lens = c.args()
    table = torch.cat([table, torch.full((3, 4), -1, dtype=torch.int32, device="cuda")], 1)
    q, ws = dev(c.q_bits), c.workspace()
    masks = c.trees(1) if tree else None
    out, lse = c.outputs()

    def call():
        if tree:
            k3.k3moe_attn_tree(c.cache, q, offs, masks, table, lens, out, lse=lse, ws=ws)
        else:
            k3.k3moe_attn_extend(c.cache, q, offs, table, lens, out, lse=lse, ws=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.fill_(9), lse.fill_(9)
    graph.replay()
    c.check(out, lse, tree=tree)
    for t, u in ((c.cache.k, d.cache.k), (c.cache.v, d.cache.v), (c.cache.k_scales, d.cache.k_scales),
                 (c.cache.v_scales, d.cache.v_scales)):
        n = min(len(t), len(u))
        t[:n], u = u[:n], None
    # the other case's tokens do not all lie in the smaller cache: only what fits is asked for
    if d.cache.pages <= c.cache.pages:
        offs.copy_(i32(d.offsets)), lens.copy_(i32(d.lens))
        table.fill_(-1)
        table[:, :d.table.shape[1]] = i32(d.table)
        q[:d.rows] = dev(d.q_bits)[:c.rows]
        out.fill_(9), lse.fill_(9)
        if tree:
            masks[:d.rows] = d.trees(1)
        graph.replay()
        d.check(out[:d.rows], lse[:d.rows], tree=tree)


def test_refusals():
    c = ExtendCase([(20, 4), (30, 5)], 4, 2, 64, 16, E4)
    q, (o, t, n), (out, lse), ws = dev(c.q_bits), c.args(), c.outputs(), c.workspace()
    m = c.trees(1)

    def fails(code, masks=None, **kw):
        a = dict(q=q, o=o, t=t, n=n, out=out, lse=lse, ws=ws) | kw
        more = {k: a[k] for k in a if k not in ("q", "o", "t", "n", "out")}
        with pytest.raises((k3.K3moeError, ValueError, TypeError)) as e:
            if masks is None:
                k3.k3moe_attn_extend(c.cache, a["q"], a["o"], a["t"], a["n"], a["out"], **more)
            else:
                k3.k3moe_attn_tree(c.cache, a["q"], a["o"], masks, a["t"], a["n"], a["out"], **more)
        if code is not None:
            assert e.value.code == code
    for masks in (None, m):
        fails(None, masks, o=o[:2])
        fails(None, masks, o=o.long())
        fails(None, masks, q=q[:, :3])
        fails(None, masks, q=q.float())
        fails(None, masks, out=out[:, :, ::2])
        fails(None, masks, lse=lse[:3])
        fails(None, masks, n=n[:1])
        fails(k3.K3MOE_ERR_SHAPE, masks, window=-1)
        fails(k3.K3MOE_ERR_SHAPE, masks, sinks=-1)
        fails(k3.K3MOE_ERR_SHAPE, masks, window=-2 ** 32)
        fails(k3.K3MOE_ERR_ARG, masks, scale=float("inf"))
        if k3.k3moe_attn_extend_workspace_bytes(c.cache, 2, c.rows, 4):
            fails(k3.K3MOE_ERR_WORKSPACE, masks, ws=None)
            fails(k3.K3MOE_ERR_WORKSPACE, masks, ws=ws[:-1])
    fails(k3.K3MOE_ERR_SHAPE, max_new=0)
    fails(None, m[:3])
    fails(None, m.int())
    fails(k3.K3MOE_ERR_SHAPE, torch.zeros(c.rows, 17, dtype=torch.int64, device="cuda"))
    out.fill_(3)
    k3.k3moe_attn_extend(c.cache, q, o, t, n, out, window=2 ** 40, sinks=2 ** 40, ws=ws)  # as without a window
    c.check(*c.run())
    none = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    k3.k3moe_attn_extend(c.cache, none, o, t, n, none)  # no rows


def test_the_same_call_gives_the_same_bits():
    c = ExtendCase([(3000, 30), (0, 300), (20, 1)], 8, 2, 128, 64, E4, seed=12)
    first = c.run(window=1000, sinks=3)
    for _ in range(5):
        again = c.run(window=1000, sinks=3)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_references():
    """The reference of a single row, by hand."""
    out, lse, _, _ = ref.attn(np.array([1.0, 0]), np.array([[0, 0], [0, 0.0]]), np.array([[1, 2], [3, 4.0]]), 1.0)
    assert np.allclose(out, [2, 3]) and np.isclose(lse, np.log(2))
