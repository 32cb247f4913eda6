"""The paged cache's upkeep on the GPU: tables, counts and lists are compared entry by entry with the
sequential definition, pages bit by bit."""
import random

import numpy as np
import pytest
import torch

from oracle import branch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF = torch.bfloat16, torch.float16


def index(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Pair:
    """A cache's tables on the device beside the definition's."""

    def __init__(self, api, B, width, pages, page, seed=0, table=None, refs=None):
        self.api, self.page, self.r = api, page, random.Random(seed)
        table = [[-1] * width for _ in range(B)] if table is None else table
        refs = [0] * pages if refs is None else refs
        self.o = branch.Cache(table, refs, page)
        self.table, self.refs = index(table), index(refs)

    def same(self, expect=0):
        assert self.api.sync_status() == expect
        assert self.table.tolist() == self.o.table
        assert self.refs.tolist() == self.o.refs

    def reserve(self, kv_len, start, tokens=None, expect=0):
        got = self.api.paged_reserve(self.table, index(kv_len), self.refs, self.page,
                                     q_start=None if start is None else index(start), tokens=tokens)
        if start is None:
            start = np.arange(0, tokens + 1, tokens // len(kv_len)).tolist()
        want = self.o.reserve(kv_len, start)
        self.same(expect)
        assert got.tolist() == want
        return got

    def fork(self, parents, kv_len=None, expect=0):
        lens = None if kv_len is None else index(kv_len)
        self.api.paged_fork(self.table, index(parents), self.refs, lens)
        want = self.o.fork(parents, kv_len)
        self.same(expect)
        assert lens is None or lens.tolist() == want
        return want

    def free(self, keep, expect=0):
        self.api.paged_free(self.table, index(keep), self.refs, self.page)
        self.o.free(keep)
        self.same(expect)

    def compact(self, expect=0):
        room = max(len(self.o.refs) // 2, 1)
        moves = torch.full((2, room + 3), -7, dtype=torch.int32, device=DEV)
        got, count = self.api.paged_compact(self.table, self.refs, moves=moves)
        src, dst = self.o.compact()
        self.same(expect)
        assert got is moves and count.tolist() == [len(src)]
        assert got.tolist() == [src + [-7] * (room + 3 - len(src)), dst + [-7] * (room + 3 - len(dst))]


# one CTA and clusters, tables wider than a block's columns, one sequence and many
@pytest.mark.parametrize("B,width,pages,page,steps", [
    (1, 1, 1, 8, 8), (1, 5, 7, 8, 20), (5, 33, 300, 16, 30), (64, 40, 9000, 8, 20), (37, 70, 33001, 32, 15),
    (700, 11, 12345, 64, 12), (1500, 3, 4099, 1024, 10), (3, 2100, 8191, 8, 15), (130, 9, 8189, 16, 12),
    (9, 40, 262145, 8, 10), (5000, 2, 9001, 64, 6), (16384, 2, 30000, 8, 5), (20, 300, 262111, 16, 8),
])
def test_random_steps_come_to_the_definitions_tables(cuda_lib, B, width, pages, page, steps):
    c = Pair(cuda_lib, B, width, pages, page, seed=B)
    r, lens, cap = c.r, [0] * B, width * page
    some = max(1, min(cap, pages * page // (3 * B)))  # so that the pool holds everyone, copies too
    for _ in range(steps):
        op = r.choice(["fork", "grow", "grow", "free", "compact"])
        if op == "fork":
            lens = c.fork([r.choice([b, b, r.randrange(B), r.randrange(B), -1]) for b in range(B)], lens)
        elif op == "grow":
            n = [min(r.choice([0, 1, 1, 2, some]), max(0, some - x)) for x in lens]
            if sum(n) == 0:
                continue
            lens = [a + b for a, b in zip(lens, n)]
            short = c.o.refs.count(0) < sum(-(-x // page) + 1 for x in n)
            if not short:
                c.reserve(lens, np.cumsum([0] + n).tolist(), tokens=sum(n) + r.choice([0, 5]))
            else:
                lens = [a - b for a, b in zip(lens, n)]
        elif op == "free":
            lens = [r.choice([x, x, 0, r.randint(0, x)]) for x in lens]
            c.free(lens)
        else:
            c.compact()


def test_every_writer_of_a_page_that_all_share(cuda_lib):
    for B in (2, 33, 1025, 9000):  # up to several rounds of every thread
        c = Pair(cuda_lib, B, 2, B + 3, 8, table=[[1, -1]] * B, refs=[0, B] + [0] * (B + 1))
        copies = c.reserve([5] * B, None, tokens=B)
        assert copies[:, 0].tolist() == [-1, -1, 0]  # the first keeps it
        assert int((copies[2] == 4).sum()) == B - 1
        c.free([5] * (B - 1) + [0])
        c.reserve([8] * B, None, tokens=B)
        held = Pair(cuda_lib, B, 2, B + 3, 8, table=[[1, -1]] * B, refs=[0, B + 1] + [0] * (B + 1))
        assert held.reserve([5] * B, None, tokens=B)[0].tolist() == [1] * B  # somebody else keeps it


def test_reserving_again_changes_nothing(cuda_lib):
    c = Pair(cuda_lib, 6, 20, 200, 16, seed=3)
    lens, start = [40, 0, 17, 16, 300, 1], [0, 40, 40, 57, 73, 373, 374]
    c.reserve(lens, start, tokens=374)
    table = c.table.clone()
    assert c.reserve(lens, start, tokens=374)[0].tolist() == [-1] * 6
    assert torch.equal(table, c.table)
    # pages reserved ahead are kept, and used
    c.reserve([60, 0, 17, 16, 300, 1], [0, 20, 20, 20, 20, 20, 20], tokens=20)
    c.reserve([45, 0, 17, 16, 300, 1], [0, 5, 5, 5, 5, 5, 5], tokens=20)


def test_as_many_tokens_for_every_sequence(cuda_lib):
    for B, each, pages in ((3, 5, 40), (40, 20, 400), (500, 33, 20000), (900, 100, 40000)):
        c = Pair(cuda_lib, B, 30, pages, 8, seed=B)
        lens = [c.r.randint(0, 60) for _ in range(B)]
        c.reserve([x + each for x in lens], None, tokens=B * each)
        c.fork([c.r.randrange(B) for _ in range(B)])
        c.free([c.r.randint(0, 100) for _ in range(B)])


def test_pages_that_the_caller_holds(cuda_lib):
    """A prefix kept by the caller: never given out, never written to, moved like the others."""
    c = Pair(cuda_lib, 3, 6, 20, 8)
    c.reserve([17, 9, 0], [0, 17, 26, 26], tokens=26)
    for e in c.o.table[0][:3]:
        c.o.refs[e] += 1
        c.refs[e] += 1
    kept = list(c.o.table[0][:3])
    c.free([0, 9, 0])
    assert [c.o.refs[e] for e in kept] == [1, 1, 1]
    c.table[2, :3] = c.table.new_tensor(kept)  # a new sequence on the kept prefix
    c.o.table[2][:3] = kept
    for e in kept:
        c.o.refs[e] += 1
        c.refs[e] += 1
    copies = c.reserve([0, 9, 18], [0, 0, 0, 1], tokens=1)  # its own copy of the part-filled page
    assert copies[:, 2].tolist() == [kept[2], c.o.table[2][2], 1]
    c.free([0, 0, 0])
    c.o.refs[kept[0]] -= 1  # the front page is given up: the others move into its place and behind
    c.refs[kept[0]] -= 1
    c.compact()
    assert sum(c.o.refs) == 2


def test_a_long_prompt_and_a_large_pool(cuda_lib):
    c = Pair(cuda_lib, 3, 20000, 100003, 8)
    c.reserve([150000, 3, 100], [0, 150000, 150003, 150103], tokens=150103)
    c.fork([2, 0, 0])
    c.reserve([101, 150001, 150009], [0, 1, 2, 11], tokens=11)
    c.free([50, 99999, 0])
    c.compact()


def test_pages_run_out(cuda_lib):
    for pages in (40, 9001):  # one CTA, a cluster
        c = Pair(cuda_lib, 4, pages, pages, 8)  # a row may name the whole pool
        most = pages * 8
        c.reserve([most - 40, 0, 0, 0], [0, most - 40] + [most - 40] * 3, tokens=most)
        # the fork's copies and the new places find fewer pages than they need: five are left
        lens = c.fork([0, 0, 0, -1], [most - 43, 0, 0, 0])
        cut = [most - 44] * 3 + [0]
        c.free(cut)
        want = [x + 30 if x else 0 for x in cut]
        c.reserve(want, [0, 30, 60, 90, 90], tokens=90, expect=cuda_lib.FA_ERR_FULL)
        assert c.o.errors == {"full"} and 0 not in c.o.refs
        c.o.errors.clear()
        # a sequence that ends makes room; what is there already stays
        c.free([want[0], 0, want[2], 0])
        assert lens[3] == 0
        c.reserve([want[0], 0, want[2], 0], [0, 30, 30, 60, 60], tokens=60,
                  expect=0 if c.o.refs.count(0) >= 8 else cuda_lib.FA_ERR_FULL)


def bad_state(api, page=8):
    """Six sequences of a table 5 wide; 30 pages, the first ten held."""
    table = [[0, 1, -1, -1, -1], [2, 3, 4, -1, -1], [2, 3, 5, -1, -1], [6, -1, -1, -1, -1], [7, 8, 9, -1, -1],
             [-1] * 5]
    refs = [0] * 30
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    return Pair(api, 6, 5, 30, page, table=table, refs=refs)


def test_values_out_of_range_are_reported_and_not_followed(cuda_lib):
    bad = cuda_lib.FA_ERR_INDEX
    c = bad_state(cuda_lib)
    c.fork([0, 6, -2, 1, 2 ** 31 - 1, -2 ** 31], [9, 20, 20, 7, 24, 0], expect=bad)
    c = bad_state(cuda_lib)
    c.free([-1, 41, 2 ** 31 - 1, -2 ** 31, 24, 0], expect=bad)
    for lens in ([16, 20, 20, 41, 25, 1], [16, 20, 20, -1, 25, 1], [16, 20, 20, 2 ** 31 - 1, 25, 1]):
        c = bad_state(cuda_lib)
        c.reserve(lens, [0, 1, 2, 3, 4, 5, 6], tokens=6, expect=bad)
        assert c.table[3].tolist() == [6, -1, -1, -1, -1]
    c = bad_state(cuda_lib)
    c.reserve([17, 20, 20, 8, 25, 1], [0, 6, 0, 6, 0, 6, 0], tokens=6, expect=bad)  # nothing at all
    c = bad_state(cuda_lib)
    c.reserve([3, 20, 20, 8, 25, 1], [0, 5, 6, 7, 8, 9, 10], tokens=10)  # tokens before a sequence: no pages
    # entries that are no pages are replaced where they are written to, and given back as nothing
    for e in (30, 2 ** 31 - 1, -2, -2 ** 31):
        c = bad_state(cuda_lib)
        c.table[1, 2] = e
        c.o.table[1][2], c.o.refs[4] = e, 0
        c.refs[4] = 0
        c.reserve([17, 20, 20, 8, 25, 1], [0, 1, 2, 3, 4, 5, 6], tokens=6, expect=bad)
        c = bad_state(cuda_lib)
        c.table[1, 2] = e
        c.o.table[1][2] = e
        c.free([0] * 6, expect=bad)
        c = bad_state(cuda_lib)
        c.table[1, 2] = e
        c.o.table[1][2] = e
        c.refs[0] = 0
        c.o.refs[0] = 0
        c.table[0, 0] = -1
        c.o.table[0][0] = -1
        c.compact(expect=bad)
    # an entry whose page nobody is said to hold
    c = bad_state(cuda_lib)
    c.refs[9] = 0
    c.o.refs[9] = 0
    c.free([0, 24, 24, 8, 0, 0], expect=bad)
    c = bad_state(cuda_lib)
    c.refs[9] = 0
    cuda_lib.paged_reserve(c.table, index([16, 24, 24, 8, 24, 0]), c.refs, 8, index([0, 0, 0, 0, 0, 1, 1]), tokens=1)
    assert cuda_lib.sync_status() == bad


def test_tables_that_do_not_start_on_a_sector(cuda_lib):
    """Rows of odd width in the middle of a larger array: what surrounds them stays."""
    buf = torch.full((4 + 5 * 7,), 77, dtype=torch.int32, device=DEV)
    table = buf[1:36].view(5, 7)
    table.fill_(-1)
    refs = torch.zeros(50, dtype=torch.int32, device=DEV)
    o = branch.Cache(table.tolist(), refs.tolist(), 8)
    lens = [9, 0, 56, 8, 1]
    cuda_lib.paged_reserve(table, index(lens), refs, 8, index([0, 9, 9, 65, 73, 74]), tokens=74)
    o.reserve(lens, [0, 9, 9, 65, 73, 74])
    cuda_lib.paged_fork(table, index([2, 2, 0, -1, 4]), refs)
    o.fork([2, 2, 0, -1, 4])
    cuda_lib.paged_free(table, index([56, 17, 9, 0, 1]), refs, 8)
    o.free([56, 17, 9, 0, 1])
    cuda_lib.paged_compact(table, refs)
    o.compact()
    assert cuda_lib.sync_status() == 0
    assert table.tolist() == o.table and refs.tolist() == o.refs
    assert buf[0].item() == 77 and buf[36:].tolist() == [77] * 3


# ------------------------------------------------------------------------------------------ copies
def pools(L, pages, heads, page, d, dtype, layout, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def bits(*shape):  # any bits: NaNs keep their payloads
        return torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device=DEV, dtype=torch.int16).view(dtype)
    if layout == "dense":
        return [bits(L, pages, heads, page, d) for _ in range(2)]
    if layout == "tokens":
        return [bits(L, pages, page, heads, d).transpose(2, 3) for _ in range(2)]
    if layout == "joint":  # K and V of a page side by side, layers inside pages, rows padded
        x = bits(pages, L, 2, heads, page, d + 8)[..., :d].transpose(0, 1)
        return [x[:, :, 0], x[:, :, 1]]
    k = bits(pages, L, heads, page, d).transpose(0, 1)  # "mixed": V a row's heads, padded
    return [k, bits(L, pages, page, heads + 1, d)[:, :, :, :heads].transpose(2, 3)]


@pytest.mark.parametrize("layout", ["dense", "tokens", "joint", "mixed"])
@pytest.mark.parametrize("L,heads,page,d,dtype", [(1, 1, 8, 64, HF), (3, 2, 16, 128, BF), (2, 7, 32, 64, BF),
                                                  (1, 8, 1024, 128, HF), (5, 1, 64, 128, BF)])
def test_copies_move_the_rows_asked_for_and_nothing_else(cuda_lib, layout, L, heads, page, d, dtype):
    r = random.Random(page + heads)
    k, v = pools(L, 23, heads, page, d, dtype, layout, seed=page)
    ids = r.sample(range(23), 18)
    src, dst = ids[:9], ids[9:]
    src[4], src[7] = src[0], -1  # one page to two, pairs left out
    dst[2] = -1
    rows = [page, 0, 5, 1, page - 1, page // 2, 3, 7, page]
    for how in (None, rows):
        want = [x.clone() for x in (k, v)]
        for w in want:
            for i, (a, b) in enumerate(zip(src, dst)):
                if a >= 0 and b >= 0:
                    n = page if how is None else how[i]
                    w[:, b, :, :n] = w[:, a, :, :n]
        cuda_lib.paged_copy(k, v, index(src), index(dst), None if how is None else index(how))
        assert cuda_lib.sync_status() == 0
        for x, w in zip((k, v), want):
            assert torch.equal(x.contiguous().view(torch.int16), w.contiguous().view(torch.int16))


def test_copies_of_one_layer_up_to_a_count(cuda_lib):
    for count, used in ((0, 0), (3, 3), (-4, 0), (99, 5)):
        k, v = (x[0] for x in pools(1, 12, 2, 16, 64, BF, "dense", seed=5))
        want = [x.clone() for x in (k, v)]
        for w in want:
            for i in range(used):
                w[6 + i] = w[i]
        cuda_lib.paged_copy(k, v, index(range(5)), index(range(6, 11)), count=index([count]))
        assert cuda_lib.sync_status() == 0
        for x, w in zip((k, v), want):
            assert torch.equal(x.view(torch.int16), w.view(torch.int16))


def test_copies_of_bad_pages_or_rows_are_left_out_and_reported(cuda_lib):
    k, v = pools(2, 9, 2, 8, 64, HF, "dense", seed=6)
    want = [x.clone() for x in (k, v)]
    for w in want:
        w[:, 8] = w[:, 0]
    src, dst, rows = [0, 1, 9, 2, 3, 2 ** 31 - 1], [8, 9, 5, 6, 7, 5], [8, 8, 8, 9, -1, 8]
    cuda_lib.paged_copy(k, v, index(src), index(dst), index(rows))
    assert cuda_lib.sync_status() == cuda_lib.FA_ERR_INDEX
    for x, w in zip((k, v), want):
        assert torch.equal(x.view(torch.int16), w.view(torch.int16))


def test_copies_behind_two_to_the_31_elements(cuda_lib):
    pages = (1 << 31) // (8 * 16 * 128) + 40
    k, v = (torch.zeros(pages, 8, 16, 128, dtype=BF, device=DEV) for _ in range(2))
    k[pages - 2], v[pages - 2] = 3.0, 5.0
    cuda_lib.paged_copy(k, v, index([pages - 2, pages - 2]), index([pages - 1, 1]))
    assert cuda_lib.sync_status() == 0
    for x, value in ((k, 3.0), (v, 5.0)):
        assert bool((x[[1, pages - 1]] == value).all()) and not bool(x[pages - 3].any() or x[0].any())


# --------------------------------------------------------------------------------- arguments, streams
def test_arguments_that_are_refused(cuda_lib):
    t, f = torch.full((3, 4), -1, dtype=torch.int32, device=DEV), torch.zeros(9, dtype=torch.int32, device=DEV)
    n = index([1, 2, 3])
    api = cuda_lib
    kv = torch.zeros(9, 2, 16, 64, dtype=BF, device=DEV)
    for call in (
            lambda: api.paged_reserve(t, n, f, 16, q_start=index([0, 1, 2, 3])),  # tokens missing
            lambda: api.paged_reserve(t, n[:2], f, 16),
            lambda: api.paged_reserve(t, n.long(), f, 16),
            lambda: api.paged_reserve(t, n, f, 16, copies=torch.zeros(2, 3, dtype=torch.int32, device=DEV)),
            lambda: api.paged_reserve(t, n, f, 16, tokens=3 << 20,
                                      workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)),
            lambda: api.paged_reserve(t[:, :3], n, f, 16),
            lambda: api.paged_fork(t, n[:2], f), lambda: api.paged_fork(t, n, f.long()),
            lambda: api.paged_fork(t, n, f[::2]), lambda: api.paged_fork(t, n, f, kv_len=n[:1]),
            lambda: api.paged_fork(t, None, f), lambda: api.paged_fork(t, n.view(3, 1).expand(3, 2), f),
            lambda: api.paged_free(t, None, f, 16),
            lambda: api.paged_free(t, n.cpu(), f, 16), lambda: api.paged_fork(t, n, None),
            lambda: api.paged_compact(t, f, moves=torch.zeros(2, 3, dtype=torch.int32, device=DEV)),
            lambda: api.paged_compact(t, f, count=f), lambda: api.paged_compact(t, f, count=f[:1].long()),
            lambda: api.paged_copy(kv, kv[:, :1], n, n), lambda: api.paged_copy(kv, None, n, n),
            lambda: api.paged_copy(kv, kv, n, n[:2]), lambda: api.paged_copy(kv, kv, n, n, rows=n[:1]),
            lambda: api.paged_copy(kv[0], kv[0], n, n), lambda: api.paged_copy(kv, kv, n, n, count=n),
            lambda: api.paged_copy(kv, kv, t, n), lambda: api.paged_copy(kv, kv, None, n)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        api.paged_copy(kv.float(), kv.float(), n, n)
    for call in (lambda: api.paged_free(t, n, torch.zeros(10, dtype=torch.int32, device=DEV)[1:], 16),  # not aligned
                 lambda: api.paged_free(t, n, f, 12), lambda: api.paged_reserve(t, n, f, 16, tokens=4),
                 lambda: api.paged_copy(kv, kv, n[:0], n[:0])):
        with pytest.raises(api.FAError):
            call()
    assert t.tolist() == [[-1] * 4] * 3 and not f.any()


def test_a_captured_step_replays_on_new_values(cuda_lib):
    """fork, reserve, copy, free and compact in one graph on another stream, against the definition."""
    B, width, pages, page, L = 6, 12, 64, 8, 2
    r = random.Random(11)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    refs, copies = torch.zeros(pages, dtype=torch.int32, device=DEV), index([[0] * B] * 3)
    moves, count = index([[-1] * (pages // 2)] * 2), index([0])
    parents, kv, start, keep = index(list(range(B))), index([0] * B), index([0] * (B + 1)), index([0] * B)
    k, v = pools(L, pages, 2, page, 64, BF, "dense", seed=12)
    side = torch.cuda.Stream()

    def step(stream=None):
        api = cuda_lib
        api.paged_fork(table, parents, refs, stream=stream)
        api.paged_reserve(table, kv, refs, page, start, tokens=24, copies=copies, stream=stream)
        api.paged_copy(k, v, copies[0], copies[1], copies[2], stream=stream)
        api.paged_free(table, keep, refs, page, stream=stream)
        api.paged_compact(table, refs, moves, count, stream=stream)
        api.paged_copy(k, v, moves[0], moves[1], count=count, stream=stream)
    torch.cuda.synchronize()
    step(side)  # allocates what a first call needs
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    o = branch.Cache(table.tolist(), refs.tolist(), page)
    data = [x.clone() for x in (k, v)]
    lens = [0] * B
    for _ in range(12):
        par = [r.choice([b, r.randrange(B), -1]) for b in range(B)]
        lens = o.fork(par, lens)
        n = [min(r.choice([0, 1, 4]), 40 - x) for x in lens]
        lens = [a + b for a, b in zip(lens, n)]
        begin = np.cumsum([0] + n).tolist()
        stay = [r.choice([x, x, r.randint(0, x)]) for x in lens]
        for x, value in ((parents, par), (kv, lens), (start, begin), (keep, stay)):
            x.copy_(index(value))
        for a, b, rows in zip(*o.reserve(lens, begin)):
            if a >= 0:
                for x in data:
                    x[:, b, :, :rows] = x[:, a, :, :rows]
        o.free(stay)
        for a, b in zip(*o.compact()):
            for x in data:
                x[:, b] = x[:, a]
        lens = stay
        torch.cuda.synchronize()
        graph.replay()
        assert cuda_lib.sync_status() == 0 and not o.errors
        assert table.tolist() == o.table and refs.tolist() == o.refs
        for x, w in zip((k, v), data):
            assert torch.equal(x.view(torch.int16), w.view(torch.int16))


def test_two_caches_on_two_streams(cuda_lib):
    """Calls of different caches may run side by side; each comes to its own definition's tables."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [Pair(cuda_lib, 40, 30, 20000, 8, seed=i) for i in range(2)]
    lens = [[10 * i + 3] * 40 for i in (1, 2)]
    args = [(index(x), index(np.arange(0, 40 * n + 1, n).tolist()), 40 * n)
            for x, n in zip(lens, (13, 23))]
    parents = [index([(7 * b + i) % 40 for b in range(40)]) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, (kv, start, T), par in zip(caches, streams, args, parents):
            cuda_lib.paged_reserve(c.table, kv, c.refs, 8, start, T, stream=s)
            cuda_lib.paged_fork(c.table, par, c.refs, stream=s)
    torch.cuda.synchronize()
    for c, x, (_, start, _), par in zip(caches, lens, args, parents):
        for _ in range(20):
            c.o.reserve(x, start.tolist())
            c.o.fork(par.tolist())
        c.same()
