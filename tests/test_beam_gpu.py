"""Beam selection on the GPU against the fp64 definition, and decoding with branches as a whole.

Tolerance of a score s = score + x - L.  The kernel's L has the errors of e^(x - m) in fp32: with
y = m - x, rounding y and y log2(e) moves a term by y (2^-24 + 2^-24) relative, the exponential by
2^-22, and sums of up to 64 terms in a row, then trees, by at most 40 roundings of 2^-24; y is weighted by the
softmax, whose mean of y is below ln V < 12.  The logarithm's mantissa adds 2^-24.  So
|dL| <= 12 2^-23 + 2^-22 + 41 2^-24 < 4.2e-6, and storing s in fp32 adds 2^-24 |s|.  Within a row the
order is exact; between rows it may differ where two scores lie within 2 |dL|.
"""
import random
import threading

import numpy as np
import pytest
import torch

from oracle import branch
from oracle import paged as op

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16, torch.float32]
DL = 4.2e-6


def check(api, logits, scores, K, finished=None, end=None, exact=True, **kw):
    """Runs the call and compares it; exact: no two scores are as close as rounding could swap."""
    B, W, V = logits.shape
    got = api.beam_select(logits, scores, k=K, finished=finished, end_token=end, **kw)
    assert api.sync_status() == 0
    s, parent, token, done = (x.cpu().numpy() for x in got)
    x, sc = logits.double().cpu().numpy(), scores.double().cpu().numpy()
    f = None if finished is None else finished.cpu().numpy()
    for b in range(B):
        want = branch.select(x[b], sc[b], K, None if f is None else f[b], -1 if end is None else end)
        there = want["beam"] >= 0
        assert np.array_equal(parent[b] >= 0, there)
        assert np.all(np.isneginf(s[b][~there])) and np.all(token[b][~there] == -1)
        beam = parent[b] - b * W
        tol = DL + 2.0 ** -24 * np.abs(want["scores"][there])
        assert np.all(np.abs(s[b][there] - want["scores"][there]) <= tol)
        if exact:
            assert np.array_equal(beam[there], want["beam"][there])
            assert np.array_equal(token[b][there], want["token"][there])
        else:  # each one is as good as the one in its place, and taken once
            c = branch.candidates(x[b], sc[b], None if f is None else f[b], -1 if end is None else end)
            mine = c[beam[there], token[b][there]]
            assert np.all(np.abs(mine - want["scores"][there]) <= 2 * DL)
            assert len(set(zip(beam[there], token[b][there]))) == there.sum()
        ended = np.ones(K, bool)
        ended[there] = token[b][there] == (-1 if end is None else end)
        if f is not None:
            ended[there] |= f[b][beam[there]] != 0
        assert np.array_equal(done[b].astype(bool), ended)
    return got


def normal(seed, *shape, dtype=torch.float32, scale=3.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def beams(seed, B, W):
    return -torch.rand(B, W, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * 9


# pieces of a row that end anywhere, all alignments, as many candidates as there are and more
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,W,V,K", [(1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 7, 21), (2, 3, 7, 30), (3, 2, 255, 4),
                                     (1, 5, 8191, 10), (2, 2, 8192, 64), (1, 3, 8193, 65), (2, 4, 20001, 8),
                                     (1, 2, 50002, 128), (5, 7, 1004, 14), (1, 40, 3001, 80),
                                     # a cluster per request up to 128 tiles in all (odd rows: 64); larger calls
                                     (77, 1, 300, 5), (80, 2, 12301, 40), (300, 1, 20002, 3), (1, 50, 30001, 9),
                                     (2, 130, 4097, 128), (64, 1, 4096, 4), (32, 2, 4100, 4), (33, 2, 4100, 4)])
def test_selection_is_the_definitions(cuda_lib, B, W, V, K, dtype):
    check(cuda_lib, normal(V + K, B, W, V, dtype=dtype), beams(V, B, W), K, exact=dtype == torch.float32)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_any_alignment_and_stride(cuda_lib, dtype):
    for off in range(9):
        big = normal(off, 3, 6, 10000 + off, dtype=dtype)
        check(cuda_lib, big[:, 1:4, off:off + 9001], beams(off, 3, 3), 6, exact=False)
    big = normal(5, 4, 2, 3000, dtype=dtype)
    check(cuda_lib, big[1::2, :, 8:2009], beams(1, 2, 2), 5, exact=False)
    # a request's beams all see the same logits
    one = normal(6, 2, 1, 9000, dtype=dtype).expand(2, 4, 9000)
    check(cuda_lib, one, beams(2, 2, 4), 8, exact=False)
    check(cuda_lib, big[:, :, :1], beams(3, 4, 2), 2, exact=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [100, 8192, 30001])
def test_equal_scores_go_by_their_place(cuda_lib, V, dtype):
    """Rows that are alike in all beams: every tie is between equal numbers, so the order is exact."""
    B, W = 2, 3
    for row in (torch.zeros(V), torch.randint(-3, 4, (V,), generator=torch.Generator().manual_seed(V)).float(),
                torch.arange(V).flip(0) // 700 * 1.0, torch.arange(V) // 900 * 1.0,
                torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)):
        x = row.to(DEV).to(dtype)[None, None].expand(B, W, V).contiguous()
        for K in (1, 7, 128):
            check(cuda_lib, x, torch.zeros(B, W, device=DEV), K)
            check(cuda_lib, x, torch.tensor([[-1.0, 0.0, 0.0], [0.0, -5.0, 0.0]], device=DEV), K)


@pytest.mark.parametrize("dtype", TYPES)
def test_ascending_and_constant_rows_take_the_bisection(cuda_lib, dtype):
    """More logits reach the bound than are ranked by counting: exact all the same."""
    V = 20000
    up = (torch.arange(V, device=DEV) % 8192 // 4).float() / 64  # four of each value
    x = torch.stack([up, up.flip(0), torch.full_like(up, 2.5), torch.full_like(up, -1e4)])[None].to(dtype)
    for K in (1, 3, 64, 100, 128):
        check(cuda_lib, x, torch.tensor([[0.0, -3.0, -11.0, -20.0]], device=DEV), K, exact=K < 5)
    # one beam alone: nothing but its own order
    for w in range(4):
        for K in (1, 64, 127):
            check(cuda_lib, x[:, w:w + 1].contiguous(), torch.zeros(1, 1, device=DEV), K)


def test_many_candidates_tie_across_beams(cuda_lib):
    """Every beam offers K equal candidates, more in all than are ranked by counting."""
    for W, V, K in ((40, 300, 128), (700, 40, 64), (2048, 3, 128)):
        x = torch.zeros(1, W, V, device=DEV)
        check(cuda_lib, x, torch.zeros(1, W, device=DEV), K)
        scores = torch.zeros(1, W, device=DEV)
        scores[0, : W // 2] = -1.0
        check(cuda_lib, x, scores, K)
        check(cuda_lib, x, scores, K, finished=(torch.arange(W, device=DEV) % 3 == 0).to(torch.uint8)[None], end=2)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_tokens_dead_beams_and_beams_that_have_ended(cuda_lib, dtype):
    B, W, V = 4, 5, 9001
    x = normal(3, B, W, V, dtype=dtype)
    allow = torch.rand(B, W, V, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)
    for share in (0.5, 0.01, 0.0002):
        y = x.masked_fill(allow >= share, float("-inf"))
        for fin in (None, torch.tensor([[0, 1, 0, 0, 255]] * B, dtype=torch.uint8, device=DEV)):
            s = beams(5, B, W)
            s[1, 0] = float("-inf")
            s[2] = float("-inf")
            check(cuda_lib, y, s, 10, fin, V - 1, exact=False)
            check(cuda_lib, y, s, 128, fin, 0, exact=False)
    check(cuda_lib, torch.full_like(x, float("-inf")), beams(6, B, W), 3)
    all_ended = torch.ones(B, W, dtype=torch.uint8, device=DEV)
    check(cuda_lib, torch.full_like(x, float("nan")), beams(7, B, W), 4, all_ended, 17)
    lowest = torch.finfo(dtype).min  # masks of the type's lowest value are logits like others
    y = x.masked_fill(allow >= 0.0002, lowest)
    check(cuda_lib, y, beams(8, B, W), 12, exact=False)
    check(cuda_lib, torch.full_like(x, lowest), torch.zeros(B, W, device=DEV), 12)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lowest", [False, True])
def test_masks_that_leave_some_tokens(cuda_lib, lowest, dtype):
    """From one token to all of them, scattered or in blocks that few threads see; the others -inf or the type's
    lowest value, whose places follow once the others run out."""
    V = 30000
    g = torch.Generator(device=DEV).manual_seed(8)
    x = normal(4, 1, 2, V, dtype=dtype)
    mask = torch.finfo(dtype).min if lowest else float("-inf")
    spread = torch.rand(V, generator=g, device=DEV).argsort()
    place = torch.arange(V, device=DEV)
    for n in (1, 7, 8, 9, 31, 100, 700, 5000):
        for block in (False, True):
            keep = (place % 2048 < 8 * n / V * 256) & (place // 8 % 3 < 2) if block else spread < n
            y = torch.where(keep, x, torch.tensor(mask, dtype=dtype, device=DEV))
            for K in (1, 8, 40, 128):
                check(cuda_lib, y, torch.tensor([[-1.0, -1.5]], device=DEV), K, exact=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [513, 848, 1024, 2000, 8192 + 600, 20000])
def test_the_best_stand_in_few_places(cuda_lib, V, dtype):
    """Short rows and ends of rows, and rows of which a range is allowed or far above the rest: few threads see all
    that reach a bound, more than there is room for.  One beam, so that the order is the logits' and exact."""
    x = normal(11, 2, 1, V, dtype=dtype)
    s = torch.tensor([[-1.0], [-2.0]], device=DEV)
    for K in (1, 9, 16, 17, 33, 64, 65, 128):
        check(cuda_lib, x, s, K)
        for lo, hi in ((0, V), (V - 600, V), (3, 520), (V // 3, V // 3 + 900), (V // 2 - 700, V // 2 + 900)):
            lo, hi = max(lo, 0), min(hi, V)
            for rest in (float("-inf"), torch.finfo(dtype).min, -20.0):
                y = torch.full_like(x, rest)
                y[..., lo:hi] = x[..., lo:hi]
                check(cuda_lib, y, s, K)
            y = x.clone()
            y[..., lo:hi] += 30
            check(cuda_lib, y, s, K)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 8191, 8192, 12344])
def test_a_row_that_is_no_distribution_offers_nothing(cuda_lib, value, at):
    x = normal(9, 2, 3, 12345)
    x[0, 1, at] = value
    x[1, 2, at] = -float("nan") if value != value else value
    s = beams(9, 2, 3)
    s[1, 0] = value
    s[1, 1] = float("nan")
    got = check(cuda_lib, x, s, 6)
    assert not bool((got[1][0] == 1).any()) and got[1][1].tolist() == [-1] * 6
    check(cuda_lib, torch.full_like(x, value), beams(1, 2, 3), 4)


def test_large_magnitudes(cuda_lib):
    for shift in (-30000.0, 0.0, 30000.0):
        x = normal(10, 2, 3, 9000) + shift
        x[..., 77] += 60.0
        check(cuda_lib, x, beams(10, 2, 3), 6, exact=False)
    # one token takes all the probability: its score is the beam's own
    x = torch.zeros(1, 2, 9000, device=DEV)
    x[0, :, 5] = 1e6
    got = check(cuda_lib, x, torch.tensor([[-2.0, -3.0]], device=DEV), 4)
    assert got[0][0, :2].tolist() == [-2.0, -3.0]


def test_results_do_not_depend_on_what_the_buffers_held(cuda_lib):
    x, s = normal(11, 80, 2, 30001, dtype=torch.bfloat16), beams(11, 80, 2)
    want = [t.clone() for t in cuda_lib.beam_select(x, s, k=9, end_token=3)]
    n = cuda_lib.beam_select_workspace_bytes(80, 2, 30001, 9)
    assert n > 0
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        out = [torch.full_like(t, 77) for t in want]
        got = cuda_lib.beam_select(x, s, k=9, end_token=3, out_scores=out[0], out_parents=out[1],
                                   out_tokens=out[2], out_finished=out[3], workspace=ws)
        assert all(a is b for a, b in zip(got, out))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert cuda_lib.sync_status() == 0


@pytest.mark.parametrize("B,W,V", [(3, 4, 3001), (70, 4, 30001), (20, 40, 3001)])
def test_scores_and_flags_in_place(cuda_lib, B, W, V):
    """A step's buffers are the next step's: also beams that have ended."""
    x, s = normal(12, B, W, V), beams(12, B, W)
    f = (torch.rand(B, W, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV) < 0.5).to(torch.uint8)
    s2, f2 = s.clone(), f.clone()
    for _ in range(3):
        want = cuda_lib.beam_select(x, s, finished=f, end_token=9)
        got = cuda_lib.beam_select(x, s2, finished=f2, end_token=9, out_scores=s2, out_finished=f2)
        assert got[0] is s2 and got[3] is f2
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        s, f = want[0], want[3]
    assert cuda_lib.sync_status() == 0


def test_beam_arguments_that_are_refused(cuda_lib):
    api, x, s = cuda_lib, normal(1, 2, 3, 50), beams(1, 2, 3)
    for call in (lambda: api.beam_select(x[0], s), lambda: api.beam_select(x, s[:1]),
                 lambda: api.beam_select(x, s.half()), lambda: api.beam_select(x, s.cpu()),
                 lambda: api.beam_select(x, None), lambda: api.beam_select(x, s, k=0),
                 lambda: api.beam_select(x, s, finished=s, end_token=1),
                 lambda: api.beam_select(x.transpose(1, 2), s),
                 lambda: api.beam_select(x, s, out_tokens=torch.zeros(2, 3, device=DEV)),
                 lambda: api.beam_select(x.repeat(300, 1, 1), s.repeat(300, 1),
                                         workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        api.beam_select(x.double(), s)
    for kw in (dict(k=129), dict(end_token=50), dict(end_token=-2),
               dict(finished=torch.zeros(2, 3, dtype=torch.uint8, device=DEV))):
        with pytest.raises(api.FAError):
            api.beam_select(x, s, **kw)


@pytest.mark.parametrize("B", [2, 60])
def test_selection_captured_and_on_two_streams(cuda_lib, B):
    xs, ss = [normal(i, B, 4, 20001, dtype=torch.float16) for i in range(3)], [beams(i, B, 4) for i in range(3)]
    want = [[t.clone() for t in cuda_lib.beam_select(x, s)] for x, s in zip(xs, ss)]
    x, s = xs[0].clone(), ss[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = cuda_lib.beam_select(x, s)
    for i in (2, 1, 0, 2):
        x.copy_(xs[i])
        s.copy_(ss[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = [[], []]
    for _ in range(20):
        for j, st in enumerate(streams):
            out[j].append(cuda_lib.beam_select(xs[j], ss[j], stream=st))
    torch.cuda.synchronize()
    for j in range(2):
        for got in out[j]:
            assert all(torch.equal(a, b) for a, b in zip(got, want[j]))
    assert cuda_lib.sync_status() == 0


def test_long_rows_and_far_requests(cuda_lib):
    """Places near 2^31 and requests further apart than 2^31 elements: zeros but for a few logits, so that the sums
    are known."""
    V = (1 << 29) + 5
    x = torch.zeros(1, 3, V, dtype=torch.bfloat16, device=DEV)
    at = [(0, 7), (0, V - 1), (1, 8191), (1, 8192), (2, V - 3), (2, 1 << 28)]
    for i, (w, v) in enumerate(at):
        x[0, w, v] = 16.0 + i
    scores = torch.tensor([[-1.0, -2.0, -4.0]], device=DEV)
    got = cuda_lib.beam_select(x, scores, k=8)
    assert cuda_lib.sync_status() == 0
    L = [np.log(V - 2 + sum(np.exp(16.0 + i) for i, (b, _) in enumerate(at) if b == w)) for w in range(3)]
    want = sorted(((float(scores[0, w]) + 16.0 + i - L[w], w, v) for i, (w, v) in enumerate(at)), reverse=True)
    low = [(float(scores[0, 0]) - L[0], 0, 0), (float(scores[0, 0]) - L[0], 0, 1)]
    want = (want + low if L[0] + 1.0 < min(L[1] + 2.0, L[2] + 4.0) else want)[:8]
    n = len(want)
    assert got[1][0, :n].tolist() == [w for _, w, _ in want] and got[2][0, :n].tolist() == [v for _, _, v in want]
    # sums of half a billion terms: up to 16 tiles of 32 in a row, then trees and 4097 pieces: 64 roundings of 2^-24
    assert np.allclose(got[0][0, :n].cpu(), [s for s, _, _ in want], rtol=2.0 ** -23, atol=2e-5)
    del x
    far = torch.empty((1 << 31) + 4096, dtype=torch.float16, device=DEV)
    y = far.as_strided((2, 2, 2000), ((1 << 31) + 8, 2001, 1))
    y.copy_(normal(3, 2, 2, 2000, dtype=torch.float16))
    check(cuda_lib, y, beams(3, 2, 2), 5, exact=False)


def test_calls_from_several_threads(cuda_lib):
    xs, ss = [normal(i, 4, 3, 5001) for i in range(4)], [beams(i, 4, 3) for i in range(4)]
    want = [[t.clone() for t in cuda_lib.beam_select(x, s)] for x, s in zip(xs, ss)]
    torch.cuda.synchronize()
    streams, wrong = [torch.cuda.Stream() for _ in range(4)], []

    def work(i):
        with torch.cuda.stream(streams[i]):
            table = torch.full((5, 9), -1, dtype=torch.int32, device=DEV)
            refs = torch.zeros(60, dtype=torch.int32, device=DEV)
            kv = torch.tensor([30, 1, 70, 8, 9], dtype=torch.int32, device=DEV)
            par = torch.tensor([2, 2, -1, 0, 4], dtype=torch.int32, device=DEV)
            o = branch.Cache(table.tolist(), refs.tolist(), 8)
            for _ in range(20):
                got = cuda_lib.beam_select(xs[i], ss[i])
                cuda_lib.paged_reserve(table, kv, refs, 8)
                cuda_lib.paged_fork(table, par, refs)
                cuda_lib.paged_compact(table, refs)
                o.reserve(kv.tolist(), list(range(6)))
                o.fork(par.tolist())
                o.compact()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])) or table.tolist() != o.table \
                        or refs.tolist() != o.refs:
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and cuda_lib.sync_status() == 0


def test_beam_search_over_the_paged_cache(cuda_lib):
    """Prompt, then steps of selection, fork, reserve, copy, append and attention, as a serving loop makes
    them; every beam's attention is compared with attention over its own history, kept apart."""
    api, d, H, Hkv, page, L, G, W, V = cuda_lib, 64, 4, 2, 8, 2, 3, 4, 300
    dtype = torch.bfloat16
    r = random.Random(5)
    S, pages = G * W, 120
    k, v = (torch.zeros(L, pages, Hkv, page, d, dtype=dtype, device=DEV) for _ in range(2))
    table = torch.full((S, 10), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    prompts = [13, 8, 21]
    n = [prompts[b // W] if b % W == 0 else 0 for b in range(S)]
    kv_len = torch.tensor(n, dtype=torch.int32, device=DEV)
    start = torch.tensor(np.cumsum([0] + n).tolist(), dtype=torch.int32, device=DEV)
    T = sum(n)
    api.paged_reserve(table, kv_len, refs, page, start, tokens=T)
    history = [[[] for _ in range(S)] for _ in range(L)]  # [layer][sequence]: (k, v) rows
    for layer in range(L):
        nk, nv = normal(layer, T, Hkv, d, dtype=dtype, scale=1.0), normal(9 + layer, T, Hkv, d, dtype=dtype, scale=1.0)
        api.paged_append(nk, nv, k[layer], v[layer], table, kv_len, start)
        for b in range(S):
            history[layer][b] = [(nk[t], nv[t]) for t in range(int(start[b]), int(start[b + 1]))]
    scores = torch.full((G, W), float("-inf"), device=DEV)
    scores[:, 0] = 0.0  # one beam each at first
    finished = torch.zeros(G, W, dtype=torch.uint8, device=DEV)
    for step in range(14):
        logits = normal(100 + step, G, W, V, dtype=dtype)
        x, sc, fin = logits.double().cpu().numpy(), scores.cpu().numpy(), finished.cpu().numpy()
        scores, parents, tokens, finished = api.beam_select(logits, scores, finished=finished, end_token=7)
        for g in range(G):
            want = branch.select(x[g], sc[g], W, fin[g], 7)
            assert np.allclose(scores[g].cpu(), want["scores"], atol=2 * DL + 1e-5)
        api.paged_fork(table, parents, refs, kv_len)
        kv_len += 1
        copies = api.paged_reserve(table, kv_len, refs, page)
        api.paged_copy(k, v, copies[0], copies[1], copies[2])
        par = parents.view(-1).tolist()
        assert min(par) >= 0
        for layer in range(L):
            nk = normal(1000 + 10 * step + layer, S, Hkv, d, dtype=dtype, scale=1.0)
            nv = normal(2000 + 10 * step + layer, S, Hkv, d, dtype=dtype, scale=1.0)
            q = normal(3000 + 10 * step + layer, S, H, d, dtype=dtype, scale=1.0)
            api.paged_append(nk, nv, k[layer], v[layer], table, kv_len)
            history[layer] = [history[layer][p] + [(nk[b], nv[b])] for b, p in enumerate(par)]
            o, lse = api.paged_attention(q, k[layer], v[layer], table, kv_len)
            if step % 4 != 1 and step != 13:
                continue
            for b in r.sample(range(S), 5):
                K = torch.stack([a for a, _ in history[layer][b]], 1).float().cpu().numpy()
                X = torch.stack([a for _, a in history[layer][b]], 1).float().cpu().numpy()
                assert int(kv_len[b]) == K.shape[1]
                ref = op.attention(q[b:b + 1].float().cpu().numpy(), K, X, d ** -0.5, K.shape[1] - 1)
                # P and O are rounded to bf16 (half a step is 2^-8 relative): two of them, with room for
                # fp32 sums of a few dozen terms
                tol = 2.0 ** -8 * (ref["absv"] + np.abs(ref["o"])) + 1e-5
                assert np.all(np.abs(o[b].float().cpu().numpy() - ref["o"][0]) <= tol[0])
                assert np.allclose(lse[b].cpu().numpy(), ref["lse"][0], atol=1e-4)
    # everything given back leaves an empty pool
    api.paged_fork(table, torch.full_like(parents, -1), refs, kv_len)
    assert api.sync_status() == 0
    assert not refs.any() and bool((table == -1).all()) and not kv_len.any()
