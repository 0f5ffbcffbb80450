"""Pins of the page book's oracle: small books worked by hand."""
import numpy as np

from oracle import kv8_pages as pages


def book(n, *rows):
    table = np.array(rows, np.int32)
    refs = np.zeros(n, np.int32)
    for p in table.flatten():
        if p >= 0:
            refs[p] += 1
    return refs, table


def test_grow_takes_the_lowest_free_pages_in_order_of_rows():
    refs, table = book(8, [6, -1, -1], [-1, 1, -1], [-1, -1, -1])
    assert pages.grow(refs, table, 16, [33, 20, 16]) == [(3, 0)]
    assert table.tolist() == [[6, 0, 2], [-1, 1, -1], [3, -1, -1]] and refs.tolist() == [1, 1, 1, 1, 0, 0, 1, 0]
    assert pages.grow(refs, table, 16, [48, 48, 48]) == [(3, 0)]          # the hole before a held entry stays
    assert table.tolist() == [[6, 0, 2], [-1, 1, 4], [3, 5, 7]]
    assert pages.grow(refs, table, 16, [48, 48, 49]) == [(0, -1)]


def test_grow_does_nothing_if_pages_are_short():
    refs, table = book(3, [2, -1, -1], [-1, -1, -1])
    assert pages.grow(refs, table, 16, [48, 16]) == [(0, 1)]
    assert table.tolist() == [[2, -1, -1], [-1, -1, -1]] and refs.tolist() == [0, 0, 1]


def test_fork_shares_full_pages_and_splits_the_last():
    refs, table = book(8, [5, 3, 7], [-1, -1, -1], [0, -1, -1])
    assert pages.fork(refs, table, 16, [0, 0, -1], [1, 2, 0], [40, 32, 5]) == [(3, 0), (7, 1), (-1, -1), (-1, -1)]
    assert table.tolist() == [[5, 3, 7], [5, 3, 1], [5, 3, -1]]
    assert refs.tolist() == [0, 1, 0, 3, 0, 3, 0, 1]
    for bad in (([0, 0], [1, 1], [1, 1]), ([0, 1], [1, 2], [1, 1]), ([0, 0], [1, 3], [1, 1]), ([0, 0], [1, 2], [1, 49])):
        assert pages.fork(refs, table, 16, *bad)[0] == (0, -1)


def test_free_by_range_and_compact():
    refs, table = book(8, [5, 3, 7], [5, 3, 1])
    pages.free(refs, table, 16, [0, 0, 9, -1], [0, 20, 0, 0], [31, 48, 99, 99])
    assert table.tolist() == [[-1, 3, -1], [5, 3, 1]] and refs.tolist() == [0, 1, 0, 2, 0, 1, 0, 0]
    assert pages.compact(refs, table, 3) == [(2, 0), (5, 0), (3, 2), (-1, -1)]
    assert table.tolist() == [[-1, 2, -1], [0, 2, 1]] and refs.tolist() == [1, 1, 2, 0, 0, 0, 0, 0]
    assert pages.compact(refs, table, 3)[0] == (0, 0)


def test_grow_deals_no_pages_for_tokens_that_a_fork_brought_along_and_lost():
    """Prefixes that end in pages their parent gave back: the child's tokens are gone, not still to come."""
    for n, entry in ((40, 2), (48, 2), (33, 2), (32, 1), (1, 0)):
        refs, table = book(20, [0, 1, 2, 3, 4, 5, 6, -1], [9, 10, -1, -1, 11, -1, -1, -1], [-1] * 8)
        pages.free(refs, table, 16, [0], [0], [48])
        assert pages.fork(refs, table, 16, [0], [1], [n]) == [(1, 0), (-1, -1)]
        want = [-1] * 8
        want[entry] = pages.GONE
        assert table[1].tolist() == want and refs.tolist() == [0, 0, 0, 1, 1, 1, 1] + [0] * 13
        assert pages.fork(refs, table, 16, [1], [2], [n]) == [(1, 0), (-1, -1)] and table[2].tolist() == want
        assert pages.grow(refs, table, 16, [0, n, n + 1]) == [(int(n % 16 == 0), 0)]
        assert pages.grow(refs, table, 16, [0, 100, 100])[0][1] == 0
        assert (table[1:, :entry + 1] < 0).all() and (table[1:, entry + 1:7] >= 0).all() and (table[1:, 7] == -1).all()
        pages.free(refs, table, 16, [1])                           # a row given back as a whole is new again
        assert pages.grow(refs, table, 16, [0, 16, 0]) == [(1, 0)]


def test_a_fork_that_ends_in_a_held_page_is_not_marked():
    refs, table = book(8, [5, 3, 7], [-1, -1, -1], [0, -1, -1])
    pages.free(refs, table, 16, [0], [0], [32])
    assert pages.fork(refs, table, 16, [0, 0], [1, 2], [48, 40]) == [(2, 0), (-1, -1), (7, 1)]       # 0: given back by this call
    assert table.tolist() == [[-1, -1, 7], [-1, -1, 7], [-1, -1, 1]]
    assert pages.fork(refs, table, 16, [0], [2], [0])[0] == (1, 0) and table[2].tolist() == [-1, -1, -1]
