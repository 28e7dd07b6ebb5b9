"""The planning oracle with pages outside the pool: no slot, a report, and nothing else changed."""
import pytest

import oracle.paged_ref as paged


@pytest.mark.parametrize("bad", [-1, 4, 0x10000001, 2 ** 31 - 1])
def test_a_page_outside_the_pool_gives_no_slot(bad):
    out, faults = paged.plan([5, 3], [1, 2], [[0, bad], [1, -1]], [2, 3, 0, 0], 0, 2, 4, 4, num_pages=4)
    assert faults == {"range"}
    assert out["slot_map"] == [-1, 7, 8, -1] and out["position"] == [5, 3, 4, 0]
    assert out["lengths"] == [6, 5] and out["block_table"] == [[0, bad], [1, 2]]
    out, faults = paged.plan([3, 3], [2, 1], [[0, -1], [1, -1]], [bad, 3, 0, 0], 0, 2, 4, 4, num_pages=4)
    assert faults == {"range"} and out["slot_map"] == [3, -1, 7, -1] and out["block_table"][0] == [0, bad]


def test_a_page_outside_the_pool_is_reported_where_it_returns():
    out, faults = paged.plan([5], [-1], [[0, 9]], [2, 3, 1, 1], 0, 2, 4, 4, num_pages=4)
    assert faults == {"range"} and out["ring"] == [2, 3, 0, 9] and out["ring_state"] == [0, 4]


def test_the_wrapped_slot_of_such_a_page_lies_in_the_pool():
    # what 32-bit arithmetic makes of page 0x10000001 at 16 tokens a page: row 1 of page 1
    wrapped = (0x10000001 * 16 + 1) % 2 ** 32
    assert wrapped == 17


@pytest.mark.parametrize("length", [9, 2 ** 31 - 1, -1])
def test_a_leaving_sequence_of_unknown_length_returns_no_page(length):
    out, faults = paged.plan([length, 3], [-1, 0], [[3, 1], [1, -1]], [0, 2, 0, 0], 0, 2, 4, 4, num_pages=4)
    assert faults == {"range"} and out["ring"] == [0, 2, 0, 0] and out["ring_state"] == [0, 2] and out["lengths"] == [0, 3]
