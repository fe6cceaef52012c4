"""GPU tests of batches with empty slots where first tokens stay visible: a row of a sequence of length 0 sees nothing, and is
no fault."""
import pytest
import torch

import mxfp4_expert_ffn_router_gb300 as k3
from extend_case import BF, E4, ExtendCase, i32
from mxfp4_expert_ffn_router_gb300 import decoder
from test_gpu_decoder_extend import H, PAGE, Model, _bf

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,sinks,rotated", [(E4, 3, True), (BF, 2, False), (E4, 0, True)])
def test_a_step_with_an_empty_row(fmt, sinks, rotated):
    m = Model(fmt, 24, sinks, rotated)
    pages = decoder.PageTable(4, 60, PAGE, 12)
    layer, live = m.layer(4), [0, 2]
    x, a = _bf(50, 4, H), None
    pages.append([0], 30), pages.append([2], 7)
    k3.k3moe_kv_write(m.cache, *(_bf(i, 37, 2, 64) for i in (8, 9)), torch.cat([pages.slots_of(b) for b in live]))
    for _ in range(3):
        new = pages.append(live)
        slots = i32([-1] * 4)
        slots[live] = new
        at = [pages.lens[b] - 1 if b in live else 0 for b in range(4)]
        x, a = layer.step(x.clone(), a, pages.table, pages.seq_lens, slots, m.at(at))
        assert layer.status.item() == 0 and torch.isfinite(x.float()).all()
        assert (layer.att[[1, 3]] == 0).all() and (layer.lse[[1, 3]] == -torch.inf).all()
    q = layer.qkv[:, :8]
    want, lse = torch.empty_like(layer.att), torch.empty_like(layer.lse)
    lens = pages.seq_lens[[0, 0, 2, 2]].contiguous()
    table = pages.table[[0, 0, 2, 2]].contiguous()
    ws = torch.empty(k3.k3moe_attn_extend_workspace_bytes(m.cache, 4, 4, 8), dtype=torch.uint8, device="cuda")
    k3.k3moe_attn_extend(m.cache, q, i32(range(5)), table, lens, want, lse=lse, window=24, sinks=sinks, max_new=1, ws=ws)
    assert torch.equal(layer.att[live], want[live]) and torch.equal(layer.lse[live], lse[live])


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("ctx", [40, 3000])
def test_rows_of_empty_sequences(ctx, fmt):
    """Their outputs are those of a row that sees nothing; lengths below 0 or past the table are faults still, and so is a row
    of a sequence of length 0 where more new tokens are allowed."""
    c = ExtendCase([(ctx, 1), (0, 1), (5, 1), (0, 1)], 8, 2, 64, 32, fmt, seed=2)
    lens = [c.lens[0], 0, c.lens[2], 0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(window=20, sinks=3, max_new=1, lens=lens, dev_status=status)
    assert status.item() == 0
    c.check(out, lse, window=20, sinks=3, rows=lambda b, i: b in (0, 2))
    assert (out[[1, 3]] == 0).all() and (lse[[1, 3]] == -torch.inf).all()
    for most, n in ((1, -1), (1, 10 ** 6), (2, 0)):
        status.zero_()
        lens[1] = n
        c.run(window=20, sinks=3, max_new=most, lens=lens, dev_status=status)
        assert status.item() == k3.K3MOE_DEV_BOUNDS


def test_masks_without_offsets_are_refused_with_sinks_too():
    m = Model(E4, 24, 3, False)
    pages = decoder.PageTable(2, 60, PAGE, 12)
    layer, slots = m.layer(2), pages.append([0, 1])
    with pytest.raises(ValueError):
        layer.attention(_bf(1, 2, H), None, pages.table, pages.seq_lens, slots, masks=torch.ones(2, 1, dtype=torch.int64, device="cuda"))
