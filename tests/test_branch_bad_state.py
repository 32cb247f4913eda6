"""The paged cache's upkeep on tables that are not as they should be: entries that are no pages, counts that are too
low.  What is reported, and the state that is left, entry by entry; the definitions on the CPU first."""
import pytest

from oracle import branch

NO_PAGES = (12, 2 ** 31 - 1, -2, -2 ** 31)


def with_entry(e):
    """Three rows, the middle one with an entry that is no page."""
    return [[0, 1, -1], [2, e, 3], [4, -1, 5]], [1, 1, 1, 1, 1, 1] + [0] * 6


# parents, whether the middle row is looked at: it goes to another row (alone, twice), is dropped, stays with a second
# child, and stays as it is
FORKS = [([0, -1, 1], True), ([1, -1, 1], True), ([0, 0, 2], True), ([1, 1, 2], True), ([2, 1, 0], False)]


@pytest.mark.parametrize("e", NO_PAGES)
@pytest.mark.parametrize("parents,seen", FORKS)
def test_oracle_fork_reports_entries_that_are_no_pages(parents, seen, e):
    table, refs = with_entry(e)
    o = branch.Cache(table, refs, 8)
    o.fork(parents)
    assert o.errors == ({"index"} if seen else set())
    assert o.table == [list(table[p]) if p >= 0 else [-1] * 3 for p in parents]
    assert all(r == sum(row.count(p) for row in o.table) for p, r in enumerate(o.refs))


# (table, refs, parents, refs afterwards, reported): pages that fewer hold than have them
LOW = [
    ([[0], [1]], [0, 1, 0], [-1, 1], [0, 1, 0], True),             # would fall to -1
    ([[0], [0], [0]], [1, 0, 0], [-1, -1, -1], [0, 0, 0], True),   # to -2
    ([[0], [0], [1]], [0, 1, 0], [0, 0, 2], [0, 1, 0], False),     # one holder less and one more: stays
    ([[0], [0], [1]], [0, 1, 0], [0, 0, 0], [1, 0, 0], False),     # one less and two more
    ([[0], [0], [0]], [1, 0, 0], [0, -1, -1], [0, 0, 0], True),
    ([[0], [1]], [-5, 1, 0], [0, 0], [0, 0, 0], True),             # was below zero already
]


@pytest.mark.parametrize("table,refs,parents,after,reported", LOW)
def test_oracle_fork_leaves_no_count_below_zero(table, refs, parents, after, reported):
    o = branch.Cache(table, refs, 8)
    o.fork(parents)
    assert o.refs == after and o.errors == ({"index"} if reported else set())


@pytest.mark.gpu
@pytest.mark.parametrize("e", NO_PAGES)
@pytest.mark.parametrize("parents,seen", FORKS)
def test_fork_reports_entries_that_are_no_pages(cuda_lib, parents, seen, e):
    from test_branch_gpu import Pair
    table, refs = with_entry(e)
    c = Pair(cuda_lib, 3, 3, len(refs), 8, table=table, refs=refs)
    c.fork(parents, [9, 20, 24], expect=cuda_lib.FA_ERR_INDEX if seen else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("table,refs,parents,after,reported", LOW)
def test_fork_leaves_no_count_below_zero(cuda_lib, table, refs, parents, after, reported):
    from test_branch_gpu import Pair
    for turn in range(20):  # whatever the order in which rows are counted
        c = Pair(cuda_lib, len(table), 1, len(refs), 8, table=table, refs=refs)
        c.fork(parents, expect=cuda_lib.FA_ERR_INDEX if reported else 0)
        assert c.refs.tolist() == after
    if parents[0] < 0:  # the page is a free one like others: given out again
        c.reserve([1] + [0] * (len(table) - 1), [0] + [1] * len(table), tokens=1)
        assert c.table[0].tolist() == [0]


@pytest.mark.gpu
def test_fork_of_many_rows_of_pages_that_nobody_is_said_to_hold(cuda_lib):
    """Blocks of all widths: counts go to zero and no further, pages given out afterwards."""
    from test_branch_gpu import Pair
    for B, width in ((40, 70), (700, 9), (3000, 3)):
        table = [[(b % 7) * width + i for i in range(width)] for b in range(B)]
        pages = 7 * width + 5
        c = Pair(cuda_lib, B, width, pages, 8, table=table, refs=[B // 12] * pages)
        c.fork([-1 if b % 4 else b for b in range(B)], expect=cuda_lib.FA_ERR_INDEX)
        assert min(c.refs.tolist()) == 0
        c.o.errors.clear()
        c.reserve([1 if b == 1 else 0 for b in range(B)], [0, 0] + [1] * (B - 1), tokens=1)
