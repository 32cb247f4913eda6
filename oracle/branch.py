"""Definitions of beam selection and of a paged cache's upkeep (test infrastructure).

Beam selection in fp64 numpy; tables and reference counts one entry at a time in plain Python.
Shares nothing with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from . import _f64


def candidates(logits, scores, finished=None, end_token: int = -1) -> np.ndarray:
    """Scores [W, V] of every continuation of one request's beams; -inf: not a candidate."""
    x = _f64(logits)
    W, V = x.shape
    out = np.full((W, V), -np.inf)
    for w in range(W):
        s = float(scores[w])
        if finished is not None and finished[w]:
            if np.isfinite(s):
                out[w, end_token] = s
            continue
        top = x[w].max()
        if not (np.isfinite(s) and np.isfinite(top)):  # a NaN, a +inf, or nothing but -inf
            continue
        out[w] = s + ((x[w] - top) - np.log(np.exp(x[w] - top).sum()))
    return out


def select(logits, scores, K: int, finished=None, end_token: int = -1) -> dict:
    """The K best of one request: scores, beam, token (-1 where none is left)."""
    c = candidates(logits, scores, finished, end_token).ravel()
    order = np.lexsort((np.arange(c.size), -c))[:K]
    order = order[np.isfinite(c[order])]
    V = logits.shape[1]
    res = {"scores": np.full(K, -np.inf), "beam": np.full(K, -1), "token": np.full(K, -1)}
    res["scores"][:order.size] = c[order]
    res["beam"][:order.size] = order // V
    res["token"][:order.size] = order % V
    return res


class Cache:
    """table [B][max_pages] and refs [num_pages] as lists; `errors` collects what would be reported."""

    def __init__(self, table, refs, page_size: int):
        self.table = [list(map(int, row)) for row in table]
        self.refs = list(map(int, refs))
        self.page = page_size
        self.errors = set()

    def real(self, e) -> bool:
        if 0 <= e < len(self.refs):
            return True
        if e != -1:
            self.errors.add("index")
        return False

    def drop(self, e):
        if self.real(e):
            if self.refs[e] > 0:
                self.refs[e] -= 1
            else:
                self.errors.add("index")

    def free(self, keep_len):
        cap = len(self.table[0]) * self.page
        for row, n in zip(self.table, keep_len):
            if not 0 <= n <= cap:
                self.errors.add("index")
            for i in range(-(-max(n, 0) // self.page), len(row)):
                self.drop(row[i])
                row[i] = -1

    def fork(self, parents, kv_len=None):
        B = len(self.table)
        if any(not -1 <= p < B for p in parents):
            self.errors.add("index")
        parents = [p if -1 <= p < B else b for b, p in enumerate(parents)]
        old = [list(row) for row in self.table]
        for b, p in enumerate(parents):
            self.table[b] = list(old[p]) if p >= 0 else [-1] * len(old[b])
        children = [0] * B
        for p in parents:
            if p >= 0:
                children[p] += 1
        changed = set()
        for b, row in enumerate(old):
            if parents[b] == b and children[b] == 1:
                continue  # not looked at
            for e in row:
                if self.real(e) and children[b] != 1:
                    self.refs[e] += children[b] - 1
                    changed.add(e)
        for e in changed:
            if self.refs[e] < 0:
                self.errors.add("index")
                self.refs[e] = 0
        if kv_len is not None:
            return [kv_len[p] if p >= 0 else 0 for p in parents]
        return None

    def reserve(self, kv_len, q_start):
        """q_start: B + 1 offsets.  Returns the copies [3][B]."""
        B, cap = len(self.table), len(self.table[0]) * self.page
        copies = [[-1] * B, [-1] * B, [0] * B]
        if any(b < a for a, b in zip(q_start, q_start[1:])):
            self.errors.add("index")
            return copies
        writing = []
        for b in range(B):
            n = q_start[b + 1] - q_start[b]
            if not 0 <= kv_len[b] <= cap:
                self.errors.add("index")
            elif n > 0 and kv_len[b] > 0:
                first = max(kv_len[b] - n, 0) // self.page
                writing += [(b, i) for i in range(first, (kv_len[b] - 1) // self.page + 1)]
        writers = {}
        for b, i in writing:
            if self.real(self.table[b][i]):
                writers.setdefault(self.table[b][i], []).append((b, i))
        keep = {w[0] for e, w in writers.items() if self.refs[e] <= len(w)}
        for e, w in writers.items():
            if self.refs[e] < len(w):  # more entries than were counted
                self.errors.add("index")
            self.refs[e] -= len(w)
        free = [e for e, r in enumerate(self.refs) if r == 0 and e not in writers]
        for b, i in writing:
            old = self.table[b][i]
            if (b, i) in keep:
                self.refs[old] = 1
                continue
            new = free.pop(0) if free else -1
            self.table[b][i] = new
            if new < 0:
                self.errors.add("full")
                continue
            self.refs[new] = 1
            ctx = max(kv_len[b] - (q_start[b + 1] - q_start[b]), 0)
            if 0 <= old < len(self.refs) and i == ctx // self.page and ctx % self.page:
                copies[0][b], copies[1][b], copies[2][b] = old, new, ctx % self.page
        return copies

    def compact(self):
        """Returns (src, dst)."""
        live = sum(r != 0 for r in self.refs)
        holes = [e for e in range(live) if self.refs[e] == 0]
        high = [e for e in range(live, len(self.refs)) if self.refs[e] != 0]
        to = dict(zip(high, holes))
        for row in self.table:
            for i, e in enumerate(row):
                if e in to:
                    row[i] = to[e]
                elif e < -1 or e >= len(self.refs) or (high and e >= high[0]):
                    self.errors.add("index")
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        return high, holes
