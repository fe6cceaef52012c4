"""GPU tests of k3moe_attn_decode's work line: items cut into pieces and joined by the
second kernel.  Only that way uses the workspace, so each case asserts by it that the
call took the line (and, where it says so, that items were cut)."""
import numpy as np
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from test_gpu_attn_decode import BF, E4, Case, _dev

pytestmark = pytest.mark.gpu
PIECES = 2 * 152  # most pieces: the workspace begins with two entries of four int32 each


def _run(c, window=0, lens=None, table=None, status=None, cut=True):
    B = len(c.lens)
    out = torch.full((B, c.Hq, c.dim), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, c.Hq), 9.0, dtype=torch.float32, device="cuda")
    ws = torch.full((k3.k3moe_attn_decode_workspace_bytes(c.cache, B, c.Hq),), 255, dtype=torch.uint8, device="cuda")
    k3.k3moe_attn_decode(c.cache, _dev(c.q_bits), torch.from_numpy(c.table if table is None else table).cuda(),
                         torch.tensor(c.lens if lens is None else lens, dtype=torch.int32, device="cuda"), out, lse=lse,
                         window=window, ws=ws, dev_status=status)
    meta = ws[:2 * PIECES * 16].view(torch.int32).view(-1, 4).cpu()
    written = (meta != -1).any(1)
    assert written.any(), "the call did not take the line"
    assert not cut or (meta[written][:, 1] > 1).any(), "no item was cut"
    return out, lse


def _lens(seed, B, most, low=1):
    lens = np.exp(np.random.default_rng(seed).uniform(np.log(low), np.log(most), B)).astype(int)
    lens[:4] = most, 0, 1, most - 1
    return lens.tolist()


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 128), (128, 32), (256, 16)])
@pytest.mark.parametrize("G", [1, 8, 9, 12, 16, 17])
def test_more_items_than_sms(fmt, dim, page, G):
    c = Case(_lens(G, 90, 1600), 2 * G, 2, dim, page, fmt, seed=dim + G)
    out, lse = _run(c)
    c.check(out, lse)
    again, lse2 = _run(c)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("G", [4, 12, 16])
def test_one_long_sequence(fmt, dim, page, G):
    c = Case([45000], G, 1, dim, page, fmt, seed=dim + G)
    c.check(*_run(c))


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("dim,G,page", [(64, 1, 16), (64, 12, 64), (128, 4, 16), (128, 16, 32), (256, 2, 64)])
def test_a_long_window_over_ragged_lengths(fmt, dim, G, page):
    c = Case(_lens(7, 90, 3000, 500), 2 * G, 2, dim, page, fmt, seed=dim + G, stale="inf")
    for window in (1501, 1100):
        c.check(*_run(c, window=window), window=window)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("dim,G", [(64, 4), (128, 12), (256, 1)])
def test_a_bad_page_inside_a_cut_item(fmt, dim, G):
    """Its 16 places count as not seen; the other sequences' bytes stay."""
    page = 16
    c = Case(_lens(9, 100, 1700), 2 * G, 2, dim, page, fmt, seed=dim)
    good, good_lse = _run(c)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    short = c.lens[0] - page
    for bad, at in ((-1, 60), (c.cache.pages, 0), (2 ** 31 - 1, 105)):
        table = c.table.copy()
        table[0, at] = bad
        st.zero_()
        out, lse = _run(c, table=table, status=st)
        assert int(st.item()) == k3.K3MOE_DEV_BOUNDS
        assert torch.equal(out[1:], good[1:]) and torch.equal(lse[1:], good_lse[1:])
        k, v, lens = c.k, c.v, c.lens
        c.k, c.v = (np.delete(x, slice(at * page, at * page + page), 0) for x in (k, v))
        c.lens = [short] + lens[1:]
        try:
            c.check(out, lse)
        finally:
            c.k, c.v, c.lens = k, v, lens


@pytest.mark.parametrize("fmt", [E4, BF])
def test_lengths_out_of_range(fmt):
    c = Case(_lens(11, 90, 1500), 24, 2, 64, 16, fmt, seed=12)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens, full = list(c.lens), c.lens
    lens[5], lens[50] = -3, -2 ** 31
    out, lse = _run(c, lens=lens, status=st)
    assert int(st.item()) == k3.K3MOE_DEV_BOUNDS
    drop = np.concatenate([np.full(n, b in (5, 50)) for b, n in enumerate(full)])
    c.lens = [max(n, 0) for n in lens]
    c.k, c.v = c.k[~drop], c.v[~drop]
    c.check(out, lse)


@pytest.mark.parametrize("fmt,G", [(E4, 4), (BF, 16)])
def test_thousands_of_sequences(fmt, G):
    """Each lane of a warp measures many sequences to find its block's piece."""
    lens = np.random.default_rng(13).integers(0, 40, 3000)
    lens[::50] = 1100
    lens[[0, 1, 2999]] = 1200, 0, 1030
    c = Case(lens.tolist(), G, 1, 64, 16, fmt, seed=14)
    c.check(*_run(c))


def test_captured_in_a_graph_follows_the_lengths():
    c = Case(_lens(15, 100, 1600), 24, 2, 128, 64, E4, seed=16)
    out = torch.empty((100, 24, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((100, 24), device="cuda")
    ws = torch.empty(k3.k3moe_attn_decode_workspace_bytes(c.cache, 100, 24), dtype=torch.uint8, device="cuda")
    q, table = _dev(c.q_bits), torch.from_numpy(c.table).cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    k3.k3moe_attn_decode(c.cache, q, table, lens, out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k3.k3moe_attn_decode(c.cache, q, table, lens, out, lse=lse, ws=ws)
    for new in (c.lens, [min(n, 65) for n in c.lens], [0] * 100, [max(n - 1, 0) for n in c.lens]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(9.0)
        ws.fill_(255)
        g.replay()
        want, wl = _run(c, lens=new, cut=False)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
