"""Rotary positions and paged caches on the CPU: the oracle's definitions, the frequency tables of
the library, and what its entry points refuse (no call here reaches a device)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import paged as op
from exact_attention_staged_gb300 import api, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


# ---------------------------------------------------------------------------- oracle definitions
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rope_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 5, 64))
    pos = rng.integers(-1000, 100000, (3, 5))
    f = op.inverse_frequencies(32)
    y = op.rope(x, pos, f, interleaved, 1.25)
    a, b = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[..., None] * f) * 1.25
    assert np.allclose(y[..., a], z.real, atol=1e-10) and np.allclose(y[..., b], z.imag, atol=1e-10)
    assert np.array_equal(y[..., 32:], x[..., 32:])


def test_oracle_rope_scores_depend_on_the_distance_alone_and_inverse_is_the_transpose():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 64))
    f = op.inverse_frequencies(64)
    s = [float((op.rope(q, [p + 7], f) * op.rope(k, [p], f)).sum()) for p in (0, 3, 500)]
    assert np.allclose(s, s[0], atol=1e-9)
    x, g = rng.standard_normal((2, 6, 64))
    p = np.arange(6) * 11
    # <g, R x> = <R^T g, x>, and the gradient of <g, R x> by differences (R is linear: exact step)
    lhs = (g * op.rope(x, p, f, True, 0.7)).sum()
    rt = op.rope(g, p, f, True, 0.7, inverse=True)
    assert abs(lhs - (rt * x).sum()) < 1e-10
    e = np.zeros_like(x)
    e[4, 9] = 1.0
    assert abs((g * op.rope(x + e, p, f, True, 0.7)).sum() - lhs - rt[4, 9]) < 1e-10


@pytest.mark.parametrize("causal", [False, True])
def test_oracle_paged_attention_is_decode_on_the_gathered_cache(causal):
    rng = np.random.default_rng(3)
    n, H, Hkv, L, d, P = 3, 4, 2, 37, 64, 8
    pages_k, pages_v = rng.standard_normal((2, 9, Hkv, P, d))
    row = rng.permutation(9)[:5]
    K, V = op.gather(pages_k, row, L), op.gather(pages_v, row, L)
    assert np.array_equal(K[:, 17], pages_k[row[2], :, 1])
    q = rng.standard_normal((n, H, d))
    got = op.attention(q, K, V, 0.3, L - n, causal)
    ref = oracle.decode(q.transpose(1, 0, 2)[None], K[None], V[None], 0.3, causal)
    assert np.allclose(got["o"], ref["o"][0].transpose(1, 0, 2), atol=1e-12)
    assert np.allclose(got["lse"], ref["lse"][0].T, atol=1e-12)


# ------------------------------------------------------------------------------ frequency tables
def units(f):
    return [int(math.ldexp(x, 64)) for x in np.asarray(f) / (2 * math.pi) % 1.0]


def test_frequency_tables_follow_their_formulas(lib):
    rot, base, s, L0 = 128, 500000.0, 8.0, 8192.0
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    want = {"plain": f, "linear": f / s, "ntk": (base * s ** (rot / (rot - 2))) ** (-2.0 * i / rot)}
    turns = L0 * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0, 1)
    want["bands"] = f * keep + f / s * (1 - keep)

    def pair(r):
        return rot * math.log(L0 / (r * 2 * math.pi)) / (2 * math.log(base))
    a, b = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
    ramp = np.clip((i - a) / (b - a), 0, 1)
    want["by_parts"] = f * (1 - ramp) + f / s * ramp
    for name, w in want.items():
        low, high = (1.0, 4.0) if name == "bands" else (1.0, 32.0)
        t, m = api.rope_frequencies(rot, base, name, s, L0, low, high)
        got = np.array([x % 2 ** 64 for x in t.tolist()], dtype=object)
        rel = max(abs(int(g) - u) / max(u, 1) for g, u in zip(got, units(w)))
        assert rel < 1e-14, name  # both round in 64-bit floating point on the way
        assert m == pytest.approx(0.1 * math.log(s) + 1 if name == "by_parts" else 1.0, rel=1e-6)
    # an integer product of the table is the angle, at positions where fp32 has lost it
    t, _ = api.rope_frequencies(rot, base)
    for p in (1, 77, 1 << 20, (1 << 31) - 1, -5):
        for j in (0, 9, 63):
            turn = (p * t[j].item()) % 2 ** 64 / 2 ** 64
            exact = math.fmod(p * float(f[j]) / (2 * math.pi), 1.0) % 1.0
            assert min(abs(turn - exact), 1 - abs(turn - exact)) < 1e-6


def test_frequency_refusals(lib):
    buf = (ctypes.c_uint64 * 64)()
    def call(rot=128, base=1e4, kind=0, factor=1.0, L0=0.0, low=0.0, high=0.0, out=buf):
        return lib.fa_rope_frequencies(out, None, rot, base, kind, factor, L0, low, high)
    assert call() == api.FA_OK
    for bad in (dict(rot=0), dict(rot=7), dict(base=1.0), dict(base=float("nan")), dict(kind=5),
                dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=2, factor=2.0, rot=2),
                dict(kind=3, factor=2.0), dict(kind=4, factor=2.0, L0=8e3, low=4.0, high=4.0),
                dict(out=None)):
        assert call(**bad) == api.FA_ERR_INVALID, bad
    with pytest.raises(ValueError):
        api.rope_frequencies(64, scaling="other")
    with pytest.raises(api.FAError):
        api.rope_frequencies(64, base=0.5)


# -------------------------------------------------------------------------------------- refusals
def test_rope_refusals(lib):
    p, n = ctypes.c_void_p(16), None

    def call(q=p, qo=p, k=n, ko=n, st=n, freq=p, pos=n, B=1, H=4, Hkv=0, N=5, d=64, rot=64, dt=1,
             ms=1.0):
        return lib.fa_rope(q, qo, k, ko, st, freq, pos, B, H, Hkv, N, d, rot, dt, 0, 0, ms, n)
    bad = [dict(q=n), dict(qo=ctypes.c_void_p(24)), dict(freq=n), dict(pos=ctypes.c_void_p(6)),
           dict(N=0), dict(B=0), dict(H=0), dict(dt=2), dict(ms=0.0), dict(ms=float("inf")),
           dict(k=p, Hkv=0), dict(k=p, ko=n, Hkv=2), dict(Hkv=2), dict(B=1 << 16, H=1 << 15),
           dict(H=1 << 16)]
    for b in bad:
        assert call(**b) == api.FA_ERR_INVALID, b
    for b in (dict(d=96), dict(rot=8), dict(rot=72), dict(rot=80, d=64), dict(rot=40)):
        assert call(**b) == api.FA_ERR_UNSUPPORTED, b
    good = [320, 80, 8, 320, 80, 8] + [0] * 6
    for i, v in ((0, -8), (1, 12), (2, 4), (3, 0), (5, 0), (0, 1 << 40)):
        st = list(good)
        st[i] = v
        assert call(B=2, st=(ctypes.c_longlong * 12)(*st)) == api.FA_ERR_INVALID, (i, v)


def paged(lib, fn, **kw):
    p = ctypes.c_void_p(16)
    a = dict(q=p, qo=p, k=p, v=p, kp=p, vp=p, o=p, lse=p, st=None, table=p, lens=p, qs=p, pos=None,
             freq=p, T=6, B=2, H=4, Hkv=2, d=64, pages=9, size=16, width=4, rot=64, dt=1, ms=1.0,
             max_q=6, scale=0.125, ws=None, wsb=0)
    a.update(kw)
    g = a.__getitem__
    if fn == "append":
        return lib.fa_paged_append(*map(g, ("q", "qo", "k", "v", "kp", "vp", "st", "table", "lens", "qs",
                                            "pos", "freq", "T", "B", "H", "Hkv", "d", "pages", "size",
                                            "width", "rot", "dt")), 0, a["ms"], None)
    return lib.fa_paged_attn(*map(g, ("q", "kp", "vp", "o", "lse", "st", "table", "lens", "qs", "T", "B",
                                      "H", "Hkv", "d", "pages", "size", "width", "max_q", "dt",
                                      "scale")), 1, a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fn", ["append", "attn"])
def test_paged_refusals(lib, fn):
    odd = ctypes.c_void_p(18)
    for b in (dict(kp=None), dict(vp=odd), dict(table=None), dict(lens=odd), dict(qs=odd), dict(T=0),
              dict(B=0), dict(Hkv=3), dict(H=0), dict(pages=0), dict(width=0), dict(dt=3),
              dict(qs=None, T=7), dict(T=1 << 29), dict(pages=1 << 28), dict(width=1 << 28)):
        assert paged(lib, fn, **b) == api.FA_ERR_INVALID, b
    for b in (dict(d=96), dict(size=4), dict(size=24), dict(size=2048)):
        assert paged(lib, fn, **b) == api.FA_ERR_UNSUPPORTED, b
    st = [256, 64] * 4 + [2048, 1024, 64] * 2 if fn == "append" else \
        [256, 64] * 2 + [2048, 1024, 64] * 2
    for i, v in ((0, 4), (3, 0), (len(st) - 3, 0), (len(st) - 1, 20), (len(st) - 4, -8)):
        bad = list(st)
        bad[i] = v
        assert paged(lib, fn, st=(ctypes.c_longlong * len(st))(*bad)) == api.FA_ERR_INVALID, (i, v)


def test_paged_refusals_of_one_call(lib):
    odd = ctypes.c_void_p(18)
    for b in (dict(k=None), dict(v=odd), dict(qo=None), dict(pos=odd), dict(ms=0.0), dict(freq=odd)):
        assert paged(lib, "append", **b) == api.FA_ERR_INVALID, b
    assert paged(lib, "append", rot=24) == api.FA_ERR_UNSUPPORTED
    for b in (dict(q=None), dict(o=odd), dict(lse=None), dict(max_q=0), dict(scale=0.0),
              dict(scale=float("nan"))):
        assert paged(lib, "attn", **b) == api.FA_ERR_INVALID, b
    assert paged(lib, "attn", H=129, Hkv=1) == api.FA_ERR_UNSUPPORTED


def test_paged_check_finds_bad_index_arrays(lib):
    table = torch.tensor([[3, 1, -1], [0, 8, 2]], dtype=torch.int32)
    lens = torch.tensor([20, 48], dtype=torch.int32)
    qs = torch.tensor([0, 4, 9], dtype=torch.int32)

    def ok(t=table, n=lens, q=qs, **kw):
        return api.paged_check(t, n, q, 9, 16, **kw)
    assert ok()                                  # the -1 lies behind the first sequence's end
    assert not ok(n=torch.tensor([33, 48], dtype=torch.int32))   # ... and now inside it
    assert not ok(n=torch.tensor([20, 49], dtype=torch.int32))   # longer than its table
    assert not ok(n=torch.tensor([-1, 48], dtype=torch.int32))
    big = table.clone()
    big[1, 1] = 9
    assert not ok(t=big)                         # no such page
    assert not ok(q=torch.tensor([0, 4, 3], dtype=torch.int32), tokens=9)
    assert not ok(q=torch.tensor([0, 4, 10], dtype=torch.int32), tokens=9)
    assert not ok(q=torch.tensor([-1, 4, 9], dtype=torch.int32))
    assert not ok(max_q=4)                       # the second brings five
    assert ok(tokens=64, max_q=5)                # a padded batch
    assert ok(q=None)                            # one token each
    assert ok(n=torch.tensor([0, 0], dtype=torch.int32))


def pieces_of(lib, seqs, Hkv, tile, tiles, causal, ctas, pad=0, page=16, width=2000):
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
    start = torch.tensor(np.cumsum([pad] + [n for n, _ in seqs]), dtype=torch.int32)
    T = max(int(start[-1]), 1) + pad
    out = np.zeros((40000, 9), dtype=np.int32)
    n = lib.fa_debug_paged_pieces(lens.data_ptr(), start.data_ptr(), T, len(seqs), Hkv, page, width, T,
                                  tile, tiles, causal, ctas, out.ctypes.data, len(out))
    assert 0 <= n <= len(out)
    return out[:n].tolist(), start.tolist()


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("seed", range(16))
def test_paged_work_is_cut_into_equal_stretches_that_cover_every_unit_once(lib, seed, causal):
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 12))
    seqs = []
    for _ in range(B):
        n = int(rng.choice([0, 1, 1, 2, 7, int(rng.integers(1, 900))]))
        seqs.append((n, max(0, n + int(rng.integers(-n, 3000)) if rng.random() < 0.3 else
                         n + int(rng.integers(0, 3000)))))
    Hkv, tile = int(rng.integers(1, 9)), int(rng.choice([1, 2, 18, 32, 42, 64, 128]))
    ctas, tiles = int(rng.choice([1, 7, 152])), int(rng.integers(1, 3))
    got, start = pieces_of(lib, seqs, Hkv, tile, tiles, causal, ctas, pad=int(rng.integers(0, 3)))
    want = []  # the line of units in order, with their key tiles and cost per tile
    unit = tile * tiles
    for b, (n, L) in enumerate(seqs):
        for g in range(Hkv):
            for i in range(0, n, unit):
                toks = min(unit, n - i)
                end = L - n + i + toks if causal else L
                want.append((b, g, start[b] + i, toks, max(1, -(-end // 128))))
    at = prev = 0
    ends = []
    for cta, b, g, tok, toks, t0, t1, count, holder in got:
        assert (b, g, tok, toks, count) == want[0] and t0 == at < t1 <= count
        # a unit's pieces stand in consecutive CTAs, and each names the one that holds the last
        assert t0 == 0 or cta == prev + 1
        prev = cta
        ends.append(holder)
        at = t1
        if t1 == count:
            assert set(ends) == {cta}
            ends = []
            want.pop(0)
            at = 0
    assert not want and at == 0
    cost = {}
    for x in got:
        c = 2 if x[4] > tile else 1
        cost[x[0]] = cost.get(x[0], 0) + c * (x[6] - x[5]) + (2 if tiles == 2 and x[5] == 0 else 0)
    if len(cost) > 2:  # shares differ by what the borders and the units' last tiles leave
        share = [cost.get(c, 0) for c in range(max(cost) + 1)]
        units = max(sum(x[0] == c for x in got) for c in cost)
        assert max(share) - min(share) <= 4 * units + 4


@pytest.mark.parametrize("n,L,Hkv,tile,causal", [(1, 2000000000, 8, 32, 1), (9000, 9000, 3, 128, 1),
                                                 (5000, 100000, 1, 16, 0), (3000, 1000, 2, 42, 1),
                                                 (1 << 20, 1 << 20, 2, 128, 1)])
def test_paged_work_of_long_sequences(lib, n, L, Hkv, tile, causal):
    got, _ = pieces_of(lib, [(1, 5), (n, L), (0, 7), (2, 300)], Hkv, tile, 2, causal, 152, page=1024,
                       width=2000000)
    for b, last in ((0, 1), (1, -(-L // 128)), (3, 3)):
        mine = [x for x in got if x[1] == b]
        units = -(-(1, n, 0, 2)[b] // (2 * tile))
        assert sum(x[5] == 0 for x in mine) == sum(x[6] == x[7] for x in mine) == units * Hkv
        assert mine[-1][6] == mine[-1][7] == max(last, 1)
    assert sorted({x[0] for x in got}) == list(range(max(x[0] for x in got) + 1))  # none idle


def test_wrappers_refuse_cpu_tensors_and_wrong_types(lib):
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError):
        api.rope(x, None, f)
    with pytest.raises(ValueError):
        api.paged_append(x[0], x[0], x, x, f, f)
    with pytest.raises(ValueError):
        api.paged_attention(x[0], x, x, f, f)
