"""The paged cache's upkeep on tables that are not as they should be: entries that are no pages, counts that are too
low.  What is reported, and the state that is left, entry by entry; the definitions on the CPU first."""
import random

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


def undercounted(B, seed):
    """B rows of two pages, the second partly filled and sometimes the row before's too; a quarter of the counts are
    zero, so that pages which are in use look free, another one less than they should be."""
    r = random.Random(seed)
    table, refs = [], [0] * (4 * B + 40)
    for b in range(B):
        row = [2 * b + 11, 2 * b + 12, -1]
        if b > 0 and r.random() < 0.3:
            row[1] = table[b - 1][1]
        table.append(row)
        for e in row[:2]:
            refs[e] += 1
    for e, n in enumerate(refs):
        refs[e] = r.choice([n, n, 0, max(n - 1, 0)])
    return table, refs


def lengths(B, seed):
    """Half of the sequences write behind their two pages, the others on the second one."""
    r = random.Random(seed)
    n = [r.choice([1, 1, 5, 0]) for _ in range(B)]
    return [13 + k if r.random() < 0.5 else 11 + k for k in n], [sum(n[:b]) for b in range(B + 1)]


def test_oracle_reserve_gives_no_page_out_that_is_written_to():
    """Page 1 is row 0's, though nobody is said to hold it: row 1 gets another one."""
    o = branch.Cache([[1], [-1]], [1, 0, 0], 8)
    copies = o.reserve([3, 1], [0, 1, 2])
    assert o.table == [[1], [2]] and o.refs == [1, 1, 1] and o.errors == {"index"}
    assert copies == [[-1, -1], [-1, -1], [0, 0]]
    for seed in range(20):
        table, refs = undercounted(30, seed)
        lens, start = lengths(30, seed)
        o = branch.Cache(table, refs, 8)
        o.reserve(lens, start)
        mine = [o.table[b][i] for b in range(30) if start[b + 1] > start[b]
                for i in range((lens[b] - start[b + 1] + start[b]) // 8, (lens[b] - 1) // 8 + 1)]
        assert len(set(mine)) == len(mine) and all(o.refs[e] >= 1 for e in mine)


# a CTA, a larger one, a cluster, and the form for any number (sequences, or pages)
@pytest.mark.gpu
@pytest.mark.parametrize("B,more", [(2, 0), (40, 0), (300, 0), (1200, 0), (3000, 0), (7000, 0), (40, 300000)])
def test_reserve_gives_no_page_out_that_is_written_to(cuda_lib, B, more):
    from test_branch_gpu import Pair, index
    for seed in range(6):
        table, refs = undercounted(B, seed)
        lens, start = lengths(B, seed)
        if start[-1] == 0:
            continue
        c = Pair(cuda_lib, B, 3, len(refs) + more, 8, table=table, refs=refs + [0] * more)
        want = branch.Cache(table, refs, 8)
        want.reserve(lens, start)
        c.reserve(lens, start, tokens=start[-1], expect=cuda_lib.FA_ERR_INDEX if want.errors else 0)
    # few pages: the last places get none
    codes = {"index": cuda_lib.FA_ERR_INDEX, "full": cuda_lib.FA_ERR_FULL}
    for seed in range(6):
        table, refs = undercounted(B, seed)
        refs = refs[:2 * B + 13]
        lens, start = [12 if b % 3 == 0 else 17 for b in range(B)], list(range(B + 1))
        c = Pair(cuda_lib, B, 3, len(refs), 8, table=table, refs=refs)
        got = cuda_lib.paged_reserve(c.table, index(lens), c.refs, 8)
        want = c.o.reserve(lens, start)
        assert cuda_lib.sync_status() in ({codes[e] for e in c.o.errors} or {0})  # the first that was met
        c.same()
        assert got.tolist() == want
