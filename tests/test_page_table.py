"""CPU tests of the decoder's page table: an append that does not fit leaves everything
as it was, so that it can be made again once pages have come back."""
import pytest

from mxfp4_expert_ffn_router_gb300.decoder import PageTable

PAGE = 16


def _state(p):
    return (list(p.lens), [list(o) for o in p.owned], list(p.free), p.table.tolist(), p.seq_lens.tolist())


def _table(lens, pages, max_pages=8):
    p = PageTable(len(lens), pages, PAGE, max_pages, device="cpu")
    for b, n in enumerate(lens):
        if n:
            p.append([b], n)
    return p


@pytest.mark.parametrize("lens,pages,which,count", [
    ([16, 16, 16], 4, [0, 1], 1),      # the second sequence
    ([16, 15], 2, [1, 0], 1),          # the first has room in its page
    ([10, 16], 2, [0], 8),             # the seventh token of one
    ([16, 16], 3, [0], 20),            # the second page of one
    ([16, 16], 3, [0, 0], 16),         # one sequence named twice
    ([0, 0], 1, [0, 1], 1)])
def test_an_append_that_does_not_fit_changes_nothing(lens, pages, which, count):
    p = _table(lens, pages)
    before = _state(p)
    with pytest.raises(RuntimeError):
        p.append(which, count)
    assert _state(p) == before


def test_a_sequence_at_its_most_pages():
    p = _table([2 * PAGE, 5], 9, max_pages=2)
    before = _state(p)
    with pytest.raises(RuntimeError):
        p.append([1, 0])
    assert _state(p) == before


def test_the_retry_returns_every_place():
    p = _table([16, 16, 16], 4)
    with pytest.raises(RuntimeError):
        p.append([0, 1])
    p.release(2)
    slots = p.append([0, 1]).tolist()
    assert p.lens == [17, 17, 0] and p.seq_lens.tolist() == [17, 17, 0]
    assert [p.slots_of(b)[-1].item() for b in (0, 1)] == slots
    assert len({s // PAGE for b in (0, 1) for s in p.slots_of(b).tolist()}) == 4


def test_an_append_that_just_fits():
    p = _table([10, 0], 3, max_pages=2)
    s = p.append([0, 1, 0], 6)  # 22 tokens of one, 6 of the other: three pages
    assert s.numel() == 18 and not p.free and p.lens == [22, 6] and p.seq_lens.tolist() == [22, 6]
    assert p.slots_of(0).tolist()[10:16] == s[:6].tolist() and p.slots_of(0).tolist()[16:] == s[12:].tolist()
    assert p.slots_of(1).tolist() == s[6:12].tolist()
    assert p.append([0], 10).numel() == 10 and p.append([]).numel() == 0
    with pytest.raises(RuntimeError):
        p.append([0])
