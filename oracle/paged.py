"""fp64 definitions of rotary positions and of attention over a paged cache (test infrastructure).

Plain numpy: one pair, one token, one row at a time where that is the definition.  Shares nothing
with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from . import _f64


def inverse_frequencies(rot: int, base: float = 10000.0) -> np.ndarray:
    """Radians per position of each of the rot / 2 pairs: base^(-2 j / rot)."""
    return base ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot)


def rope(x, pos, inv_freq, interleaved: bool = False, mscale: float = 1.0,
         inverse: bool = False) -> np.ndarray:
    """Rotary positions: x [..., d], pos broadcastable to x.shape[:-1].

    Pair j, elements (j, j + r/2) or (2j, 2j + 1) of the first r = 2 len(inv_freq), is multiplied by
    the matrix mscale * [[cos t, -sin t], [sin t, cos t]] with t = pos * inv_freq[j] (its transpose
    with ``inverse``); the other elements stay.
    """
    y = _f64(x).copy()
    f = np.asarray(inv_freq, dtype=np.float64)
    r = 2 * len(f)
    p = np.broadcast_to(np.asarray(pos, dtype=np.float64), y.shape[:-1])
    for j in range(r // 2):
        a, c = (2 * j, 2 * j + 1) if interleaved else (j, j + r // 2)
        t = p * f[j]
        co, si = np.cos(t) * mscale, np.sin(t) * mscale * (-1.0 if inverse else 1.0)
        ya, yc = y[..., a].copy(), y[..., c].copy()
        y[..., a] = co * ya - si * yc
        y[..., c] = si * ya + co * yc
    return y


def gather(pages, table_row, length: int) -> np.ndarray:
    """[H_kv, length, d]: the first `length` positions of a sequence whose pages table_row names."""
    pages = _f64(pages)
    _, heads, size, d = pages.shape
    out = np.empty((heads, length, d))
    for pos in range(length):
        out[:, pos] = pages[int(table_row[pos // size]), :, pos % size]
    return out


def attention(q, keys, values, scale: float, n_ctx: int, causal: bool = True) -> dict:
    """Rows q [n, H, d] of one sequence over its keys and values [H_kv, L, d].

    Row i stands at position n_ctx + i and sees keys j <= n_ctx + i (causal) or all L.  Returns o
    [n, H, d], lse [n, H], absv = sum_j P_j |v_j| (what a relative error of the probabilities can
    move o by), qk = max_j scale sum |q||k_j| over visible keys (what rounding a score goes by),
    vsum = e^(max s - lse) sum_j |v_j| (what an absolute error of probabilities that are relative
    to the largest can move o by).  A row that sees no key has o = 0, lse = -inf.
    """
    q, keys, values = _f64(q), _f64(keys), _f64(values)
    n, H, d = q.shape
    heads, L, _ = keys.shape
    rep = H // heads
    res = {"o": np.zeros((n, H, d)), "lse": np.full((n, H), -np.inf), "absv": np.zeros((n, H, d)),
           "qk": np.zeros((n, H)), "vsum": np.zeros((n, H, d))}
    for h in range(H):
        K, V = keys[h // rep], values[h // rep]
        for i in range(n):
            end = min(L, n_ctx + i + 1) if causal else L
            if end <= 0:
                continue
            s = scale * (K[:end] @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            l = e.sum()
            res["o"][i, h] = (e @ V[:end]) / l
            res["lse"][i, h] = m + np.log(l)
            res["absv"][i, h] = (e @ np.abs(V[:end])) / l
            res["qk"][i, h] = scale * (np.abs(K[:end]) @ np.abs(q[i, h])).max()
            res["vsum"][i, h] = np.abs(V[:end]).sum(0) / l
    return res
