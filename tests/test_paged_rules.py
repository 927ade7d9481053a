"""Which requests of one call are served when free pages run out: the rule by hand, on the oracle here and
on the device in the GPU tests."""
import numpy as np

import oracle.paged as op


def shortage():
    """(lens, n_pages, adds, starts, lens after) of a reservation: pages of 4, two of them free.

    Request 0 takes one of the two free pages.  1 needs two and is refused; 2 needs one, and with 0 and 1
    that makes four: refused, though a page is free.  3 and 4 need none and are served."""
    return [4, 4, 4, 2, 0], 6, [4, 8, 1, 2, 0], [4, -1, -1, 2, 0], [8, 4, 4, 4, 0]


def bad_position():
    """(lens, n_pages, keep_pos, keep_n, ok) of a compaction: pages of 4, three of them free.

    Request 0 keeps a position outside its sequence and is refused, but its two pages still count: 1, which
    needs two, is refused, though three are free.  2 needs no page and is served."""
    pos = np.zeros((1, 3, 1, 6), np.int32)
    pos[0, :, 0] = np.arange(6)
    pos[0, 0, 0, 5] = 8
    return [8, 8, 4], 8, pos, [6, 5, 0], [0, 0, 1]


def table_of(lens, n_pages, ps=4, width=4):
    table, refs, at = np.full((len(lens), width), -1, np.int32), np.zeros(n_pages, np.int32), 0
    for s, n in enumerate(lens):
        for j in range(-(-n // ps)):
            table[s, j] = at
            refs[at] = 1
            at += 1
    return table, refs


def _oracle(lens, n_pages):
    k = np.arange(n_pages * 4, dtype=np.float64).reshape(1, n_pages, 1, 4, 1)
    table, refs = table_of(lens, n_pages)
    return op.Pages(k, -k, table, np.array(lens, np.int32), refs)


def test_requests_behind_a_shortage():
    lens, n_pages, add, start, after = shortage()
    o = _oracle(lens, n_pages)
    assert o.reserve(list(range(5)), add).tolist() == start and o.lens.tolist() == after
    assert o.refs.tolist() == [1, 1, 1, 1, 1, 0]
    assert o.reserve([2], [1]).tolist() == [4]           # by itself it is served


def test_requests_behind_a_bad_position():
    lens, n_pages, pos, keep, ok = bad_position()
    o = _oracle(lens, n_pages)
    assert o.compact([0, 1, 2], pos, keep).tolist() == ok
    assert o.lens.tolist() == [8, 8, 0] and o.refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 0]
    assert o.compact([1], pos[:, 1:2], keep[1:2]).tolist() == [1]
