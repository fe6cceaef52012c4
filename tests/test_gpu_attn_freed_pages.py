"""GPU tests of k3moe_attn_decode with a window over pages that have been given back:
table entries of pages that lie wholly before the window name no page, and the call is
valid: status 0, and the bytes that the full table gives."""
import numpy as np
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from test_gpu_attn_decode import BF, E4, Case

pytestmark = pytest.mark.gpu


def _freed(c, page, window, entry):
    table = c.table.copy()
    for b, n in enumerate(c.lens):
        table[b, :max(0, n - window) // page] = entry
    return table


def _same_with_freed_pages(c, page, window):
    out, lse = c.run(window=window)
    c.check(out, lse, window=window)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for entry in (-1, c.cache.pages, 2 ** 31 - 1):
        got, gl = c.run(window=window, table=_freed(c, page, window, entry), status=st)
        assert int(st.item()) == 0, entry
        assert torch.equal(got, out) and torch.equal(gl, lse), entry


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 32), (128, 16), (256, 16), (128, 32), (64, 128)])
@pytest.mark.parametrize("window", [1, 16, 17, 33, 100, 500])
def test_short_calls(fmt, dim, page, window):
    c = Case([1, 700, 0, 64, 500, 33, 1050, 32], 6, 2, dim, page, fmt, seed=window + dim)
    _same_with_freed_pages(c, page, window)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 16)])
def test_many_short_items(fmt, dim, page):
    lens = np.random.default_rng(3).integers(0, 120, 600)
    lens[0] = 120
    c = Case(lens.tolist(), 4, 2, dim, page, fmt, seed=4)
    _same_with_freed_pages(c, page, 45)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 32), (128, 16)])
def test_long_calls(fmt, dim, page):
    lens = np.random.default_rng(5).integers(0, 4000, 60)
    lens[:3] = 4000, 0, 1501
    c = Case(lens.tolist(), 4, 4, dim, page, fmt, seed=6)
    _same_with_freed_pages(c, page, 1501)


def test_a_page_inside_the_window_is_still_reported():
    """The page that holds the window's first place is needed, with one tile before that place or none."""
    for window in (17, 16, 32):
        c = Case([48], 2, 2, 64, 16, E4, seed=7)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        table = _freed(c, 16, window, -1)
        table[0, (48 - window) // 16] = -1
        c.run(window=window, table=table, status=st)
        assert int(st.item()) == k3.K3MOE_DEV_BOUNDS, window
