"""Beam selection and the paged cache's upkeep on the CPU: the oracle's definitions, what the entry
points refuse (no call here reaches a device), and the Python checks."""
import ctypes
import random

import numpy as np
import pytest
import torch

from oracle import branch
from exact_attention_staged_gb300 import api, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


# ---------------------------------------------------------------------------- oracle definitions
def test_oracle_selection_is_a_sorted_list_of_log_probabilities():
    rng = np.random.default_rng(1)
    x, s = rng.standard_normal((3, 7)) * 4, np.array([-1.0, -2.5, -0.5])
    got = branch.select(x, s, 21)
    p = np.exp(x) / np.exp(x).sum(1, keepdims=True)
    every = sorted(((s[w] + np.log(p[w, v]), -w * 7 - v) for w in range(3) for v in range(7)), reverse=True)
    assert np.allclose(got["scores"], [e[0] for e in every])
    assert (got["beam"] * 7 + got["token"]).tolist() == [-e[1] for e in every]
    # the candidates of a beam sum to its own probability
    assert np.allclose(np.exp(branch.candidates(x, s)).sum(1), np.exp(s))


def test_oracle_selection_at_its_edges():
    x = np.zeros((2, 4))
    assert branch.select(x, [0.0, 0.0], 5)["token"].tolist() == [0, 1, 2, 3, 0]  # equals in order
    x[0, 1], x[1, 2] = np.nan, np.inf
    assert branch.select(x, [0.0, 0.0], 2)["beam"].tolist() == [-1, -1]
    x = np.full((2, 4), -np.inf)
    x[1, 3] = 5.0
    got = branch.select(x, [0.0, -1.0], 2)
    assert got["scores"].tolist() == [-1.0, -np.inf] and got["token"].tolist() == [3, -1]
    got = branch.select(x, [-9.0, -np.inf], 2, finished=[1, 0], end_token=2)
    assert got["scores"].tolist() == [-9.0, -np.inf] and got["token"].tolist() == [2, -1]


def holders(c):
    n = [0] * len(c.refs)
    for row in c.table:
        for e in row:
            if e >= 0:
                n[e] += 1
    return n


@pytest.mark.parametrize("seed", range(6))
def test_oracle_cache_keeps_its_counts_and_its_contents(seed):
    """Every token of every sequence, followed by value through forks, copies and moves."""
    r = random.Random(seed)
    B, width, P, page = r.randint(2, 7), 12, 60, r.choice([2, 4])
    c = branch.Cache([[-1] * width for _ in range(B)], [0] * P, page)
    data = [[None] * page for _ in range(P)]
    want = [[] for _ in range(B)]
    for step in range(60):
        op = r.choice(["fork", "grow", "grow", "free", "compact"])
        if op == "fork":
            parents = [r.choice([b, b, r.randrange(B), -1]) for b in range(B)]
            lens = c.fork(parents, [len(x) for x in want])
            want = [list(want[p]) if p >= 0 else [] for p in parents]
            assert lens == [len(x) for x in want]
        elif op == "grow":
            n = [min(r.choice([0, 1, 1, 3]), width * page - len(x)) for x in want]
            if sum(-(-len(x) // page) + 2 for x in want) > P:
                continue
            copies = c.reserve([len(x) + k for x, k in zip(want, n)], np.cumsum([0] + n).tolist())
            for a, b, rows in zip(*copies):
                if a >= 0:
                    data[b][:rows] = data[a][:rows]
            for b in range(B):
                for _ in range(n[b]):
                    pos, token = len(want[b]), (step, b, r.random())
                    assert c.refs[c.table[b][pos // page]] == 1
                    data[c.table[b][pos // page]][pos % page] = token
                    want[b].append(token)
        elif op == "free":
            keep = [r.choice([len(x), len(x), r.randint(0, len(x))]) for x in want]
            c.free(keep)
            want = [x[:n] for x, n in zip(want, keep)]
        else:
            src, dst = c.compact()
            for a, b in zip(src, dst):
                data[b] = list(data[a])
            live = sum(x > 0 for x in c.refs)
            assert all(x > 0 for x in c.refs[:live]) and not any(c.refs[live:])
        assert c.refs == holders(c) and not c.errors
        for row, x in zip(c.table, want):
            assert [data[row[i // page]][i % page] for i in range(len(x))] == x


def test_oracle_cache_hands_a_page_to_its_first_writer_when_all_write():
    c = branch.Cache([[0, -1], [0, -1], [0, -1]], [3, 0, 0, 0], 4)
    copies = c.reserve([3, 3, 3], [0, 1, 2, 3])
    assert [row[0] for row in c.table] == [0, 1, 2] and c.refs == [1, 1, 1, 0]
    assert copies == [[-1, 0, 0], [-1, 1, 2], [0, 2, 2]]
    c = branch.Cache([[0], [0], [0]], [3, 0, 0, 0], 4)  # the third only reads: both writers leave
    assert c.reserve([3, 3, 2], [0, 1, 2, 2])[0] == [0, 0, -1]
    assert [row[0] for row in c.table] == [1, 2, 0] and c.refs == [1, 1, 1, 0]


# -------------------------------------------------------------------------------------- refusals
P16, ODD, NONE = ctypes.c_void_p(16), ctypes.c_void_p(18), None


def reserve(lib, table=P16, lens=P16, qs=P16, refs=P16, copies=P16, T=6, B=2, pages=9, size=16, width=4,
            ws=P16, wsb=1 << 20):
    return lib.fa_paged_reserve(table, lens, qs, refs, copies, T, B, pages, size, width, ws, wsb, None)


def test_reserve_refusals(lib):
    for b in (dict(table=NONE), dict(table=ODD), dict(lens=NONE), dict(lens=ODD), dict(qs=ODD),
              dict(refs=NONE), dict(refs=ctypes.c_void_p(24)), dict(copies=ODD), dict(T=0), dict(B=0),
              dict(pages=0), dict(width=0), dict(qs=NONE, T=7), dict(B=9000, ws=NONE),
              dict(B=9000, ws=ctypes.c_void_p(8)), dict(B=9000, wsb=255), dict(pages=1 << 28), dict(width=1 << 28), dict(T=1 << 30)):
        assert reserve(lib, **b) == api.FA_ERR_INVALID, b
    for b in (dict(size=4), dict(size=24), dict(size=2048), dict(B=16385, T=16385)):
        assert reserve(lib, **b) == api.FA_ERR_UNSUPPORTED, b
    assert api.paged_reserve_workspace_bytes(64, 2, 100, 16) == 0
    assert api.paged_reserve_workspace_bytes(8192, 300, 100000, 8) == 0  # 1024 + 2 * 300 places in 8 CTAs
    assert api.paged_reserve_workspace_bytes(1 << 20, 300, 1000, 8) == ((1 << 17) + 600) * 4 // 256 * 256 + 256
    assert api.paged_reserve_workspace_bytes(300, 300, 300000, 8) == 600 * 4 // 256 * 256 + 256  # a large pool
    assert api.paged_reserve_workspace_bytes(0, 1, 100, 16) == 0


def test_fork_free_and_compact_refusals(lib):
    def fork(table=P16, lens=NONE, parents=P16, refs=P16, B=2, pages=9, width=4):
        return lib.fa_paged_fork(table, lens, parents, refs, B, pages, width, None)

    def free(table=P16, keep=P16, refs=P16, B=2, pages=9, size=16, width=4):
        return lib.fa_paged_free(table, keep, refs, B, pages, size, width, None)

    def compact(table=P16, refs=P16, src=P16, dst=P16, count=P16, B=2, pages=9, width=4):
        return lib.fa_paged_compact(table, refs, src, dst, count, B, pages, width, None)
    both = (dict(table=NONE), dict(table=ODD), dict(refs=NONE), dict(refs=ODD), dict(B=0), dict(pages=0),
            dict(width=0), dict(pages=1 << 28), dict(width=1 << 28))
    for fn, more in ((fork, (dict(parents=NONE), dict(parents=ODD), dict(lens=ODD))),
                     (free, (dict(keep=NONE), dict(keep=ODD))),
                     (compact, (dict(src=NONE), dict(dst=ODD), dict(count=NONE), dict(src=ODD)))):
        for b in both + more:
            assert fn(**b) == api.FA_ERR_INVALID, (fn.__name__, b)
        assert fn(B=16385) == api.FA_ERR_UNSUPPORTED
    for size in (4, 24, 2048):
        assert free(size=size) == api.FA_ERR_UNSUPPORTED


def test_copy_refusals(lib):
    def copy(k=P16, v=P16, st=NONE, src=P16, dst=P16, rows=NONE, count=NONE, n=3, L=2, heads=2, d=64, pages=9,
             size=16):
        return lib.fa_paged_copy(k, v, st, src, dst, rows, count, n, L, heads, d, pages, size, None)
    for b in (dict(k=NONE), dict(v=ctypes.c_void_p(24)), dict(src=NONE), dict(dst=NONE), dict(src=ODD),
              dict(rows=ODD), dict(count=ODD), dict(n=0), dict(L=0), dict(heads=0), dict(pages=0)):
        assert copy(**b) == api.FA_ERR_INVALID, b
    for b in (dict(d=96), dict(size=4), dict(size=12)):
        assert copy(**b) == api.FA_ERR_UNSUPPORTED, b
    good = [20000, 2048, 1024, 64] * 2
    for i, x in ((0, 0), (1, 4), (3, -8), (6, 20), (7, 0), (4, 1 << 40)):
        st = list(good)
        st[i] = x
        assert copy(st=(ctypes.c_longlong * 8)(*st)) == api.FA_ERR_INVALID, (i, x)


def test_beam_refusals(lib):
    def beam(x=P16, st=NONE, scores=P16, fin=NONE, os=P16, op=P16, ot=P16, of=P16, B=2, W=3, V=50, K=3,
             dt=api.FA_BF16, end=-1, ws=P16, wsb=1 << 20):
        return lib.fa_beam_select(x, st, scores, fin, os, op, ot, of, B, W, V, K, dt, end, ws, wsb, None)
    odd = ctypes.c_void_p(17)
    for b in (dict(x=NONE), dict(x=odd), dict(x=ODD, dt=api.FA_FP32), dict(scores=NONE), dict(scores=ODD),
              dict(os=NONE), dict(op=ODD), dict(ot=NONE), dict(of=NONE), dict(B=0), dict(W=0), dict(V=0),
              dict(K=0), dict(dt=3), dict(dt=-1), dict(end=50), dict(end=-2), dict(fin=P16),
              dict(B=600, ws=NONE), dict(B=600, ws=ODD), dict(B=600, wsb=16), dict(W=2000, V=1 << 21),
              dict(B=1 << 22, W=1 << 10), dict(st=(ctypes.c_longlong * 2)(-1, 50)), dict(st=(ctypes.c_longlong * 2)(150, 1 << 40))):
        assert beam(**b) == api.FA_ERR_INVALID, b
    for b in (dict(K=129), dict(W=2049)):
        assert beam(**b) == api.FA_ERR_UNSUPPORTED, b
    assert api.beam_select_workspace_bytes(2, 3, 50, 3) == 0  # done in one launch
    # 256 rows of 32 tiles of 4096 logits in two pieces each: 512 lists of 8 candidates, and sums
    assert api.beam_select_workspace_bytes(64, 4, 131072, 8) == 512 * 8 * 8 + 512 * 8
    assert api.beam_select_workspace_bytes(0, 3, 50, 3) == 0
    assert api.beam_select_workspace_bytes(2, 3, 50, 129) == 0


def test_new_constants_match_the_header(lib):
    from test_abi import header_constants
    consts = header_constants()
    for name in ("FA_FP32", "FA_ERR_INDEX", "FA_ERR_FULL"):
        assert getattr(api, name) == consts[name], name
    assert "free pages" in api.status_string(api.FA_ERR_FULL)


def test_wrappers_refuse_cpu_tensors(lib):
    x, i = torch.zeros(2, 3, 5), torch.zeros(2, 4, dtype=torch.int32)
    for call in (lambda: api.beam_select(x, x[..., 0]), lambda: api.paged_fork(i, i[:, 0], i[0]),
                 lambda: api.paged_free(i, i[:, 0], i[0], 16), lambda: api.paged_compact(i, i[0]),
                 lambda: api.paged_reserve(i, i[:, 0], i[0], 16),
                 lambda: api.paged_copy(x, x, i[0], i[0])):
        with pytest.raises(ValueError):
            call()
