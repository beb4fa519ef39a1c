"""The page state's rules on the host, on states small enough to follow by hand: pages
of 16 rows, one array whose row r holds the byte r."""
import numpy as np
import pytest

from oracle import attn as A


def _pages(batch, width, num):
    return A.Pages(np.full((batch, width), -1, np.int32), np.zeros(batch, np.int32), np.zeros(batch, np.int32),
                   np.zeros(num, np.int32), 16, [np.arange(16 * num, dtype=np.uint8)[:, None]])


def _forked(num=4):
    """Two sequences on the 10 rows of page 0."""
    s = _pages(2, 3, num)
    slots, short = s.reserve([10, 0], 10)
    assert short == 0 and slots[0].tolist() == list(range(10)) and (slots[1] == -1).all()
    s.compact(None, [10, 0], slots)
    s.fork([(0, 1)])
    assert s.table[:, 0].tolist() == [0, 0] and s.refs.tolist() == [2] + [0] * (num - 1) and s.lens.tolist() == [10, 10]
    return s


@pytest.mark.parametrize("accepted", [None, np.array([[2, 0, 1]] * 2)])
def test_a_refused_reservation_commits_nothing(accepted):
    s = _forked(num=2)                                  # copies would take two pages, one is free
    slots, short = s.reserve([3, 3], 3)
    assert short == 1 and (slots == -1).all()
    s.compact(accepted, [3, 3], slots)
    assert s.lens.tolist() == [10, 10] and s.arrays[0][:, 0].tolist() == list(range(32))


def test_sharers_that_reserve_commit_into_their_copies():
    s = _forked()
    slots, short = s.reserve([3, 2], 3)
    assert short == 0 and slots.tolist() == [[26, 27, 28], [42, 43, -1]] and s.refs.tolist() == [0, 1, 1, 0]
    assert s.arrays[0][16:26, 0].tolist() == s.arrays[0][32:42, 0].tolist() == list(range(10))
    s.compact(np.array([[2, 0, 0], [1, 0, 0]]), [2, 3], slots)          # of sequence 1 only two were reserved
    assert s.lens.tolist() == [12, 12]
    assert s.arrays[0][26:29, 0].tolist() == [28, 26, 28] and s.arrays[0][42:44, 0].tolist() == [43, 42]
    s.compact(None, [1, 1], slots)                      # these slots have been committed
    assert s.lens.tolist() == [12, 12]


def test_sharers_that_commit_without_a_reservation_move_nothing_in_one_call():
    s = _forked()
    s.compact(np.array([[3, 1], [4, 2]]), [2, 2])
    assert s.lens.tolist() == [12, 12] and s.arrays[0][:, 0].tolist() == list(range(64))
    s = _forked()                                       # one of them alone: the other's tokens end before
    s.compact(np.array([[3, 1], [4, 2]]), [1, 0])
    assert s.lens.tolist() == [11, 10] and s.arrays[0][10, 0] == 13


def test_entries_outside_the_pool_are_skipped():
    s = _forked()
    s.table[0, 0] = 4
    slots, short = s.reserve([3, 3], 3)
    assert short == 0 and slots.tolist() == [[-1, -1, -1], [26, 27, 28]]
    s.compact(None, [3, 3], slots)
    assert s.lens.tolist() == [10, 13]
    s.free([0, 1])
    assert s.refs.tolist() == [1, 0, 0, 0] and (s.table == -1).all()    # page 0: the entry that is gone held it
