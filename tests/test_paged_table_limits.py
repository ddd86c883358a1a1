"""The page table at sizes that whole numbers of 64 or 32 bits do not hold, without a GPU."""
import numpy as np
import pytest
import torch

import bit_post_quantized_smooth_amd as sq
from test_paged_table import check, same, state


@pytest.mark.parametrize("counts", [[2 ** 63 - 1, 1], [1, 2 ** 63 - 1], [2 ** 62, 2 ** 62], [2 ** 63 - 1, 2 ** 63 - 1], 2 ** 63 - 1,
                                    [65, 0], np.array([2 ** 64 - 1, 0], np.uint64)])
def test_counts_whose_sums_wrap_change_nothing(counts):
    t = sq.PageTable(2, 64, page_size=16, device="cpu")
    t.begin([3, 16])
    before, free, tables = state(t), list(t._free), t._tables.copy()
    with pytest.raises(ValueError, match="tokens|counts|sequences"):
        t.begin(counts)
    assert same(before, state(t)) and t._free == free and np.array_equal(t._tables, tables)
    assert [t.length(0), t.length(1)] == [3, 16]
    t.begin(1)
    check(t)


@pytest.mark.parametrize("a,match", [(dict(capacity=2 ** 26 + 1, pages=4, step_tokens=1), "2\\^26"), (dict(capacity=64, pages=-1), "pages"),
                                     (dict(capacity=64, page_size=1024, pages=2 ** 21 + 1), "2\\^31"),
                                     (dict(capacity=64, step_tokens=-1), "step_tokens")])
def test_tables_beyond_the_operators_refused(a, match):
    """Slots are int32, and attention takes up to 2^26 keys of a sequence."""
    with pytest.raises(ValueError, match=match):
        sq.PageTable(1, device="cpu", **a)


def test_the_last_slot_of_the_largest_pool():
    t = sq.PageTable(1, 1024, page_size=1024, pages=2 ** 21, device="cpu")
    t._free = [2 ** 21 - 1]
    t.begin(1024)
    assert int(t.slots[1023]) == 2 ** 31 - 1 and int(t.slots[0]) == 2 ** 31 - 1024
