"""CPU tests of the positions of new tokens where a sequence is named more than once, as append allows."""
import pytest

from mxfp4_expert_ffn_router_gb300.decoder import PageTable

PAGE = 16


@pytest.mark.parametrize("which,count", [([0, 0], 1), ([1, 0, 1], 2), ([0, 1, 1, 0, 0], 3), ([1], 5), ([], 2), ([0, 0], 0)])
def test_positions_in_the_order_of_the_slots(which, count):
    p = PageTable(2, 20, PAGE, 8, device="cpu")
    p.append([0], 40), p.append([1], 5)
    slots = p.append(which, count).tolist()
    at = p.positions_of(which, count).tolist()
    assert slots == [p.slots_of(b).tolist()[x] for b, x in zip([b for b in which for _ in range(count)], at)]
    assert len(at) == len(which) * count


@pytest.mark.parametrize("which,count", [([1], 6), ([1, 1], 3), ([0], -1)])
def test_more_than_there_are(which, count):
    p = PageTable(2, 20, PAGE, 8, device="cpu")
    p.append([0], 40), p.append([1], 5)
    with pytest.raises(ValueError):
        p.positions_of(which, count)
