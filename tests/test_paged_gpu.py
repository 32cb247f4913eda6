"""GPU parity of the paged cache (fa_paged_append, fa_paged_attn) with the fp64 definitions.

Append: a row of K as in test_rope_gpu (same tolerance); V and everything not named by a token is
bitwise unchanged.

Attention, element by element, derived:
  * a score is a sum of d products of 16-bit values in fp32, then a multiply-add and a 2^x: with
    delta = 2^-18 (1 + max_j scale sum |q||k_j|) its exponential and the normalisation by the sum
    are each off by less than delta relative, so O by 2 delta sum_j P_j |v_j|;
  * the probabilities are rounded to 16 bits before they meet V: eps / 2 relative each, so O by
    eps / 2 sum_j P_j |v_j|; fp16 probabilities below 2^-14 lose half of 2^-24 absolute while the
    row's largest is at least 1: 2^-25 e^(max s - lse) sum_j |v_j|;
  * O is rounded once: eps / 2 |O|.
LSE: delta plus 2^-20 (1 + |lse|) for the logarithm and the final conversion.
"""
import numpy as np
import pytest
import torch

from oracle import paged as op

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Batch:
    """A paged batch: `seqs` is a list of (new tokens, cached positions with them)."""

    def __init__(self, seqs, H, Hkv, d, dtype, page, rows=False, seed=0, pad=(0, 0), poison=True,
                 room=0):
        g = torch.Generator().manual_seed(1000 + seed)
        self.seqs, self.H, self.Hkv, self.d, self.page = seqs, H, Hkv, d, page
        B = len(seqs)
        need = [-(-L // page) for _, L in seqs]
        pool = sum(need) + 2
        ids = torch.randperm(pool, generator=g).tolist()
        # behind a sequence's pages the table holds ids that no call may follow
        width = max(max(need) + 1, -(-room // page))
        self.table = torch.full((B, width), 1 << 20, dtype=torch.int32)
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = torch.tensor(ids[at:at + c], dtype=torch.int32)
            at += c
        self.pool = pool
        shape = (pool, page, Hkv, d) if rows else (pool, Hkv, page, d)
        self.k = torch.randn(shape, generator=g).to(dtype)
        self.v = torch.randn(shape, generator=g).to(dtype)
        if rows:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        if poison:  # whatever lies behind a sequence's end has no influence
            keep = torch.zeros(pool, page, dtype=torch.bool)
            for b, (_, L) in enumerate(seqs):
                for i in range(need[b]):
                    keep[int(self.table[b, i]), :min(page, L - i * page)] = True
            for x in (self.k, self.v):
                x.masked_fill_(~keep[:, None, :, None], float("nan"))
        self.lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
        n = [m for m, _ in seqs]
        self.start = torch.tensor(np.cumsum([pad[0]] + n), dtype=torch.int32)
        self.T = pad[0] + sum(n) + pad[1]
        self.q = torch.randn((self.T, H, d), generator=g).to(dtype)
        self.max_q = max(n)
        if poison and sum(pad):
            self.q[:pad[0]] = float("nan")
            self.q[pad[0] + sum(n):] = float("nan")

    def dev(self):
        return tuple(x.to(DEV) for x in (self.q, self.k, self.v, self.table, self.lens, self.start))


def attend(api, t, scale=None, causal=True, **kw):
    q, k, v, table, lens, start = t.dev()
    if "max_q" not in kw:
        kw["max_q"] = t.max_q
    return api.paged_attention(q, k, v, table, lens, start, scale=scale, causal=causal, **kw)


def check(t, o, lse, scale, causal, what=""):
    eps = torch.finfo(o.dtype).eps
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    tiny = 2.0 ** -25 if eps < 2.0 ** -8 else 0.0
    for b, (n, L) in enumerate(t.seqs):
        if n == 0:
            continue
        K, V = op.gather(t.k, t.table[b], L), op.gather(t.v, t.table[b], L)
        at = int(t.start[b])
        r = op.attention(t.q[at:at + n], K, V, scale, L - n, causal)
        delta = 2.0 ** -18 * (1 + r["qk"])
        bound = (2 * delta[..., None] + eps / 2) * r["absv"] + tiny * r["vsum"]
        bound += eps / 2 * (np.abs(r["o"]) + bound) + tiny
        err = np.abs(o[at:at + n] - r["o"])
        assert (err <= bound).all(), f"{what} sequence {b}: O off by {(err - bound).max():.3e} beyond"
        none = np.isneginf(r["lse"])
        assert np.array_equal(np.isneginf(lse[at:at + n]), none), f"{what} sequence {b}: -inf rows"
        lerr = np.abs(lse[at:at + n][~none] - r["lse"][~none])
        lb = (delta + 2.0 ** -20 * (1 + np.abs(np.where(none, 0, r["lse"]))))[~none]
        assert (lerr <= lb).all(), f"{what} sequence {b}: LSE"


BF, HF = torch.bfloat16, torch.float16
CASES = [  # sequences (new, length), H, Hkv, d, dtype, page size, token rows outside heads, causal
    ([(1, 1)], 1, 1, 64, BF, 16, False, True),
    ([(1, 300)], 8, 2, 128, BF, 16, False, True),
    ([(1, 127), (1, 128), (1, 129), (1, 5), (1, 1000)], 4, 1, 128, HF, 32, False, True),
    ([(1, 640)] * 7, 6, 2, 64, BF, 64, True, True),
    ([(4, 500), (1, 77), (3, 3), (2, 260)], 7, 1, 64, HF, 8, False, True),
    ([(5, 1500)], 16, 16, 128, BF, 128, True, True),
    ([(70, 70), (1, 900), (130, 400)], 4, 2, 128, BF, 16, False, True),
    ([(300, 300)], 3, 1, 64, HF, 256, False, True),
    ([(257, 1100), (0, 50), (64, 64), (0, 0), (1, 33)], 8, 1, 128, BF, 32, True, True),
    ([(90, 250), (1, 40), (7, 513)], 6, 3, 64, BF, 1024, False, False),
    ([(33, 129), (200, 777)], 5, 5, 128, HF, 64, True, False),
    ([(2, 40)], 128, 1, 128, BF, 16, False, True),
    ([(600, 700)], 10, 2, 64, BF, 128, False, True),
    ([(1, 4100), (1, 65)], 32, 8, 128, BF, 16, False, True),
]


# room: positions that the tables could hold; batches whose tables hold few positions may be computed
# by clusters of CTAs, the others as one line of work over the chip
@pytest.mark.parametrize("room", [0, 9000])
@pytest.mark.parametrize("seqs,H,Hkv,d,dtype,page,rows,causal", CASES)
def test_attention_parity(cuda_lib, seqs, H, Hkv, d, dtype, page, rows, causal, room):
    t = Batch(seqs, H, Hkv, d, dtype, page, rows, seed=len(seqs) + H + d, room=room)
    o, lse = attend(cuda_lib, t, causal=causal)
    assert cuda_lib.sync_status() == 0
    check(t, o, lse, d ** -0.5, causal, "parity")
    # T as the bound on the new tokens is slower, never different
    o2, lse2 = attend(cuda_lib, t, causal=causal, max_q=None)
    check(t, o2, lse2, d ** -0.5, causal, "loose bound")


@pytest.mark.parametrize("lens", [[1], [100] * 3, [129, 500, 1, 64, 1000], [600] * 16, [40] * 40,
                                  [4000, 20], [5100], [0, 7, 0, 300]])
@pytest.mark.parametrize("n", [1, 3])
def test_short_and_few_sequences(cuda_lib, lens, n):
    # from one unit to more units than SMs, key tiles fewer and more than the CTAs that share them
    for H, Hkv, d, dtype in ((4, 1, 128, BF), (8, 4, 64, HF), (16, 8, 128, BF)):
        t = Batch([(min(n, L), L) if L else (0, 0) for L in lens], H, Hkv, d, dtype, 16, seed=sum(lens))
        o, lse = attend(cuda_lib, t)
        assert cuda_lib.sync_status() == 0
        check(t, o, lse, d ** -0.5, True, f"few {lens} {H} {Hkv} {d}")
        again = attend(cuda_lib, t)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("seqs", [[(50, 50)], [(300, 700)], [(200, 210), (1, 90), (64, 64)], [(33, 20)],
                                  [(0, 5), (130, 600), (2, 2)], [(500, 500)]])
@pytest.mark.parametrize("H,Hkv,d,dtype", [(4, 1, 128, BF), (3, 1, 64, HF), (4, 2, 64, BF), (7, 1, 128, HF)])
def test_short_chunks(cuda_lib, seqs, H, Hkv, d, dtype):
    # chunks whose units a cluster takes: units of one and of two query tiles, tiles of uneven reach,
    # fewer key tiles than CTAs
    t = Batch(seqs, H, Hkv, d, dtype, 16, seed=60 + H)
    for causal in (True, False):
        o, lse = attend(cuda_lib, t, causal=causal)
        assert cuda_lib.sync_status() == 0
        check(t, o, lse, d ** -0.5, causal, f"chunk {seqs} {H} {Hkv} {d}")


@pytest.mark.parametrize("room", [0, 9000])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_that_see_nothing_and_sharp_scores(cuda_lib, dtype, room):
    # fewer tokens than a query tile, some of them before their sequence
    t = Batch([(5, 3), (1, 0), (6, 140), (2, 1)], 4, 2, 64, dtype, 16, seed=15, room=room)
    o, lse = attend(cuda_lib, t)
    assert cuda_lib.sync_status() == 0
    check(t, o, lse, 0.125, True, "short few")
    assert bool((o[:2] == 0).all()) and bool(torch.isneginf(lse[5]).all())
    t = Batch([(2, 900), (1, 700)], 4, 2, 64, dtype, 32, seed=16, room=room)
    t.q *= 5
    o, lse = attend(cuda_lib, t, scale=1.0)
    check(t, o, lse, 1.0, True, "sharp few")
    # more new tokens than positions: the first rows stand before the sequence and see no key
    t = Batch([(9, 4), (150, 20), (3, 0), (1, 0), (140, 141)], 4, 2, 64, dtype, 16, seed=5, room=room)
    o, lse = attend(cuda_lib, t)
    assert cuda_lib.sync_status() == 0
    check(t, o, lse, 0.125, True, "short")
    assert bool((o[:5] == 0).all()) and bool(torch.isneginf(lse[:5]).all())
    # scores of std 40: nearly one-hot rows, the running maximum moves by far more than 8
    t = Batch([(40, 800), (1, 900)], 4, 2, 64, dtype, 32, seed=6, room=room)
    t.q *= 5
    o, lse = attend(cuda_lib, t, scale=1.0)
    check(t, o, lse, 1.0, True, "sharp")


def test_padded_batch_leaves_foreign_rows_alone(cuda_lib):
    t = Batch([(3, 40), (0, 9), (20, 200)], 4, 2, 128, BF, 16, seed=7, pad=(2, 5))
    out = torch.full((t.T, 4, 128), 3.0, dtype=BF, device=DEV)
    lse = torch.full((t.T, 4), 3.0, device=DEV)
    attend(cuda_lib, t, out=out, lse=lse)
    check(t, out, lse, 128 ** -0.5, True, "padded")
    for x in (out, lse):
        assert bool((x[:2] == 3.0).all()) and bool((x[-5:] == 3.0).all())
    assert cuda_lib.sync_status() == 0


def test_strided_rows_uniform_batches_and_shared_pages(cuda_lib):
    t = Batch([(2, 50)] * 3, 4, 2, 64, BF, 16, seed=8)
    q, k, v, table, lens, start = t.dev()
    want = cuda_lib.paged_attention(q, k, v, table, lens, start, max_q=2)
    joint = torch.zeros(t.T, 12, 64, dtype=BF, device=DEV)
    joint[:, 3:7] = q
    room = torch.zeros(t.T, 9, 64, dtype=BF, device=DEV)
    got = cuda_lib.paged_attention(joint[:, 3:7], k, v, table, lens, None, out=room[:, 1:5])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((room[:, 0] == 0).all()) and bool((room[:, 5:] == 0).all())
    # one pool for K and V, pages of the two side by side
    pool = torch.stack((k, v), 1)
    got = cuda_lib.paged_attention(q, pool[:, 0], pool[:, 1], table, lens, start)
    assert torch.equal(got[0], want[0])
    # every sequence reads the first one's pages
    same = table[:1].repeat(3, 1)
    a = cuda_lib.paged_attention(q[:2].repeat(3, 1, 1), k, v, same, lens, start, max_q=2)[0]
    assert torch.equal(a[2:4], a[:2]) or torch.allclose(a[2:4].float(), a[:2].float(), atol=2e-2)


@pytest.mark.parametrize("rows", [False, True])
def test_pools_with_padding_between_rows_heads_and_pages(cuda_lib, rows):
    # no stride is a multiple of the one inside it
    t = Batch([(2, 70), (40, 300)], 4, 2, 64, BF, 16, seed=18, rows=rows)
    q, k, v, table, lens, start = t.dev()
    want = cuda_lib.paged_attention(q, k, v, table, lens, start, max_q=40)
    P, H, S, d = k.shape
    row, head, page = (2 * 72 + 8, 72, 16 * 152 + 40) if rows else (72, 16 * 72 + 24, 2 * 1176 + 56)
    pad = []
    for x in (k, v):
        room = torch.full((P * page,), 9.0, dtype=BF, device=DEV)
        y = torch.as_strided(room, (P, H, S, d), (page, head, row, 1))
        y.copy_(x)
        pad.append(y)
    got = cuda_lib.paged_attention(q, pad[0], pad[1], table, lens, start, max_q=40)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    new = torch.randn(t.T, 2, 64, device=DEV).to(BF)
    cuda_lib.paged_append(new, new, k, v, table, lens, start)
    cuda_lib.paged_append(new, new, pad[0], pad[1], table, lens, start)
    assert torch.equal(pad[0].nan_to_num(), k.nan_to_num())
    assert torch.equal(pad[1].nan_to_num(), v.nan_to_num())
    assert cuda_lib.sync_status() == 0
    with pytest.raises(cuda_lib.FAError):  # K and V order heads and rows differently
        other = v.transpose(1, 2).contiguous().transpose(1, 2) if not rows else v.contiguous()
        cuda_lib.paged_attention(q, k, other, table, lens, start)
    with pytest.raises(cuda_lib.FAError):  # a broadcast Q
        cuda_lib.paged_attention(q[:1].expand(t.T, 4, 64), k, v, table, lens, start)


def test_refusals_on_device(cuda_lib):
    t = Batch([(2, 70)], 4, 2, 64, BF, 16, seed=19)
    q, k, v, table, lens, start = t.dev()
    good = dict(q=q, k_pages=k, v_pages=v, block_table=table, kv_len=lens, q_start=start)
    for bad in (dict(q=q.half()), dict(q=q[0]), dict(k_pages=k[:1]), dict(block_table=table.long()),
                dict(block_table=table[:, ::2]), dict(kv_len=lens.cpu()), dict(kv_len=lens.float()),
                dict(q_start=start[:1]), dict(out=q[:1]), dict(out=q.half()),
                dict(lse=torch.zeros(2, 4, dtype=torch.float64, device=DEV)), dict(k_pages=None),
                dict(lse=torch.zeros(4, 2, device=DEV).t())):
        with pytest.raises((ValueError, TypeError, AttributeError)):
            cuda_lib.paged_attention(**{**good, **bad})
    wide = torch.zeros(1, 1000, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):  # too small a workspace
        cuda_lib.paged_attention(**{**good, "block_table": wide},
                                 workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    for bad in (dict(max_q=0), dict(scale=0.0), dict(scale=float("inf"))):
        with pytest.raises(cuda_lib.FAError):
            cuda_lib.paged_attention(**{**good, **bad})
    x = q[:, :2]
    good = dict(k=x, v=x, k_pages=k, v_pages=v, block_table=table, kv_len=lens, q_start=start)
    f, _ = cuda_lib.rope_frequencies(64, device=DEV)
    for bad in (dict(k=q), dict(v=x[:1]), dict(q=q[:, :, :32]), dict(out_q=q), dict(freq=f.int()),
                dict(positions=lens), dict(q=q, out_q=q[:1]), dict(freq=f.cpu())):
        with pytest.raises((ValueError, TypeError)):
            cuda_lib.paged_append(**{**good, **bad})
    assert cuda_lib.sync_status() == 0


def test_calls_from_several_threads(cuda_lib):
    import threading
    batches = [Batch([(1, 900 + 100 * i), (60, 400)], 4, 2, 64, BF, 16, seed=70 + i, room=9000 * (i % 2))
               for i in range(4)]
    dev = [b.dev() for b in batches]
    want = [cuda_lib.paged_attention(*x, max_q=60) for x in dev]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        side = torch.cuda.Stream()
        for _ in range(30):
            o, lse = cuda_lib.paged_attention(*dev[i], max_q=60, stream=side)
        side.synchronize()
        if not (torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])):
            bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not bad and cuda_lib.sync_status() == 0


@pytest.mark.parametrize("room", [0, 9000])
def test_bad_indices_are_reported_not_followed(cuda_lib, room):
    t = Batch([(2, 100), (3, 50)], 4, 2, 64, BF, 16, seed=9, poison=False, room=room)
    q, k, v, table, lens, start = t.dev()
    good = cuda_lib.paged_attention(q, k, v, table, lens, start, max_q=3)
    assert cuda_lib.sync_status() == 0
    for entry in (-1, t.pool, 1 << 30):
        bad = table.clone()
        bad[0, 2] = entry
        o, _ = cuda_lib.paged_attention(q, k, v, bad, lens, start, max_q=3)
        assert cuda_lib.sync_status() == cuda_lib.FA_ERR_INDEX
        assert bool(torch.isfinite(o).all())
    for wrong in (dict(lens=torch.tensor([100, 1 << 20], dtype=torch.int32, device=DEV)),
                  dict(lens=torch.tensor([-4, 50], dtype=torch.int32, device=DEV)),
                  dict(start=torch.tensor([0, 2, 99], dtype=torch.int32, device=DEV)), dict(max_q=2)):
        a = dict(lens=lens, start=start, max_q=3)
        a.update(wrong)
        cuda_lib.paged_attention(q, k, v, table, a["lens"], a["start"], max_q=a["max_q"])
        assert cuda_lib.sync_status() == cuda_lib.FA_ERR_INDEX, wrong
    again = cuda_lib.paged_attention(q, k, v, table, lens, start, max_q=3)
    assert torch.equal(again[0], good[0]) and cuda_lib.sync_status() == 0


@pytest.mark.parametrize("room", [0, 9000])
@pytest.mark.parametrize("seqs", [[(1, 300), (2, 500)], [(300, 700)]])
def test_timeout_is_reported_not_hung(cuda_lib, seqs, room):
    t = Batch(seqs, 4, 2, 64, BF, 16, seed=17, room=room)
    want = attend(cuda_lib, t)
    assert cuda_lib.sync_status() == 0
    try:
        cuda_lib.debug_set_wait_limit_ns(20_000_000)
        cuda_lib.debug_set_fault(4)
        attend(cuda_lib, t)
        assert cuda_lib.sync_status() == cuda_lib.FA_ERR_TIMEOUT
    finally:
        cuda_lib.debug_set_fault(0)
        cuda_lib.debug_set_wait_limit_ns(0)
    got = attend(cuda_lib, t)
    assert torch.equal(got[0], want[0]) and cuda_lib.sync_status() == 0


def test_repeats_streams_graphs_and_two_calls_at_once(cuda_lib):
    t = Batch([(1, 3000), (40, 900), (1, 70)], 8, 2, 128, BF, 16, seed=10)
    q, k, v, table, lens, start = t.dev()
    a = dict(max_q=40)
    want = cuda_lib.paged_attention(q, k, v, table, lens, start, **a)
    nbytes = cuda_lib.paged_workspace_bytes(t.T, 3, 8, 2, 128, 40, 16, table.shape[1])
    ws = [torch.full((max(nbytes, 16),), 255, dtype=torch.uint8, device=DEV) for _ in range(2)]
    for _ in range(3):  # a poisoned workspace, and again with what the last call left in it
        got = cuda_lib.paged_attention(q, k, v, table, lens, start, workspace=ws[0], **a)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    t2 = Batch([(1, 500), (40, 2000), (1, 7)], 8, 2, 128, BF, 16, seed=11)
    u = t2.dev()
    want2 = cuda_lib.paged_attention(*u, **a)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):  # two calls in flight, each with a workspace of its own
        outs.append((cuda_lib.paged_attention(q, k, v, table, lens, start, stream=sides[0], **a), want))
        outs.append((cuda_lib.paged_attention(*u, stream=sides[1], **a), want2))
    torch.cuda.synchronize()
    assert all(torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]) for x, y in outs)
    # captured once, replayed on other lengths, tokens and pages; two graphs share a workspace
    o, l = torch.zeros_like(q), torch.zeros(t.T, 8, device=DEV)
    graphs = []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            cuda_lib.paged_attention(q, k, v, table, lens, start, out=o, lse=l, workspace=ws[0], **a)
    t3 = Batch([(40, 2900), (1, 1000), (1, 50)], 8, 2, 128, BF, 16, seed=12)
    w = t3.dev()
    pages = min(k.shape[0], w[1].shape[0])
    keep = [x.clone() for x in (q, k, v, table, lens, start)]
    q.copy_(w[0])
    k[:pages].copy_(w[1][:pages])
    v[:pages].copy_(w[2][:pages])
    table.fill_(0)
    m = min(table.shape[1], w[3].shape[1])
    table[:, :m] = w[3][:, :m].clamp(max=pages - 1)
    lens.copy_(w[4])
    start.copy_(w[5])
    ref = cuda_lib.paged_attention(q, k, v, table, lens, start, **a)
    for g in graphs + graphs:
        o.zero_()
        g.replay()
        assert torch.equal(o, ref[0]) and torch.equal(l, ref[1])
    for x, y in zip((q, k, v, table, lens, start), keep):
        x.copy_(y)
    graphs[0].replay()
    assert torch.equal(o, want[0])


def test_cache_beyond_32_bit_offsets(cuda_lib):
    # 2^31 elements in K alone; the sequence's pages stand at the pool's end
    page, Hkv, d = 128, 8, 128
    pool = (1 << 31) // (page * Hkv * d) + 8
    k = torch.empty(pool, Hkv, page, d, dtype=BF, device=DEV)
    v = torch.empty_like(k)
    t = Batch([(2, 300)], 8, Hkv, d, BF, page, seed=13, poison=False)
    last = [pool - 1, pool - 5, pool - 2]
    for i, p in enumerate(last):
        k[p] = t.k[int(t.table[0, i])].to(DEV)
        v[p] = t.v[int(t.table[0, i])].to(DEV)
    table = torch.tensor([last], dtype=torch.int32, device=DEV)
    o, lse = cuda_lib.paged_attention(t.q.to(DEV), k, v, table, t.lens.to(DEV))
    check(t, o, lse, d ** -0.5, True, "far pages")
    new = torch.randn(2, Hkv, d, device=DEV).to(BF)
    cuda_lib.paged_append(new, new, k, v, table, t.lens.to(DEV))
    assert torch.equal(k[pool - 2, :, 42:44].transpose(0, 1), new)
    assert cuda_lib.sync_status() == 0


# ---------------------------------------------------------------------------------------- append
APPEND = [  # sequences, H (0: no Q), Hkv, d, rot, interleaved, dtype, page, token rows
    ([(1, 1)], 2, 1, 64, 64, False, BF, 16, False),
    ([(1, 17), (1, 16), (1, 300)], 8, 2, 128, 128, False, BF, 16, False),
    ([(5, 5), (0, 9), (33, 100), (1, 64)], 3, 3, 64, 32, True, HF, 8, True),
    ([(40, 200), (2, 2)], 0, 2, 128, 48, False, HF, 64, False),
    ([(200, 201)], 7, 1, 128, 96, True, BF, 1024, True),
    ([(6, 4), (3, 0)], 4, 2, 64, 16, False, BF, 16, False),  # rows that stand before the sequence
    ([(1, 9 + i) for i in range(70)], 4, 1, 64, 64, False, BF, 16, False),
]


@pytest.mark.parametrize("seqs,H,Hkv,d,rot,inter,dtype,page,rows", APPEND)
@pytest.mark.parametrize("turned", [True, False])
def test_append_parity(cuda_lib, seqs, H, Hkv, d, rot, inter, dtype, page, rows, turned):
    from test_rope_gpu import near
    t = Batch(seqs, max(H, 1), Hkv, d, dtype, page, rows, seed=30 + H, pad=(1, 3), poison=False)
    g = torch.Generator().manual_seed(31)
    joint = torch.randn((t.T, H + 2 * Hkv, d), generator=g).to(dtype)
    dj = joint.to(DEV)
    q, k, v = dj[:, :H], dj[:, H:H + Hkv], dj[:, H + Hkv:]
    _, kp, vp, table, lens, start = t.dev()
    table_f, _ = cuda_lib.rope_frequencies(rot, device=DEV)
    out = torch.full((t.T, H, d), 5.0, dtype=dtype, device=DEV) if H else None
    got = cuda_lib.paged_append(k, v, kp, vp, table, lens, start, q=q if H else None, out_q=out,
                                freq=table_f if turned else None, interleaved=inter, mscale=0.75)
    assert cuda_lib.sync_status() == 0 and (got is out)
    f = op.inverse_frequencies(rot)
    ref_k, ref_v = t.k.clone(), t.v.clone()
    seen = torch.zeros(t.k.shape[0], page, dtype=torch.bool)
    for b, (n, L) in enumerate(seqs):
        for i in range(n):
            tok, pos = int(t.start[b]) + i, L - n + i
            if turned and H:
                near(out[tok], joint[tok, :H], op.rope(joint[tok, :H], pos, f, inter, 0.75), rot, inter,
                     0.75, "q")
            elif H:
                assert torch.equal(out[tok].cpu(), joint[tok, :H])
            if pos < 0:
                continue
            p, r = int(t.table[b, pos // page]), pos % page
            seen[p, r] = True
            x = joint[tok, H:H + Hkv]
            if turned:
                near(kp[p, :, r], x, op.rope(x, pos, f, inter, 0.75), rot, inter, 0.75, "k")
                ref_k[p, :, r] = kp[p, :, r].cpu()
            else:
                ref_k[p, :, r] = x
            ref_v[p, :, r] = joint[tok, H + Hkv:]
    assert torch.equal(kp.cpu(), ref_k) and torch.equal(vp.cpu(), ref_v)
    if H:  # tokens of no sequence
        assert bool((out[0] == 5.0).all()) and bool((out[-3:] == 5.0).all())


def test_append_positions_in_place_and_bad_pages(cuda_lib):
    t = Batch([(3, 20), (2, 40)], 4, 2, 64, BF, 16, seed=40, poison=False)
    g = torch.Generator().manual_seed(41)
    q, k, v = (torch.randn((5, h, 64), generator=g).to(BF).to(DEV) for h in (4, 2, 2))
    _, kp, vp, table, lens, start = t.dev()
    f, _ = cuda_lib.rope_frequencies(64, device=DEV)
    pos = torch.tensor([5, 900, 31, 7, 8], dtype=torch.int32, device=DEV)
    want_q, want_k = cuda_lib.rope(q.transpose(0, 1)[None], k.transpose(0, 1)[None], f, pos[None])
    cuda_lib.paged_append(k, v, kp, vp, table, lens, start, q=q, out_q=q, freq=f, positions=pos)
    assert torch.equal(q, want_q[0].transpose(0, 1))
    row = t.table[1, 2]
    assert torch.equal(kp[int(row), :, 6:8], want_k[0][:, 3:5])
    assert cuda_lib.sync_status() == 0
    before = kp.clone(), vp.clone()
    for entry in (-1, t.pool, 1 << 30):
        bad = table.clone()
        bad[0, 1] = bad[1, 2] = entry
        cuda_lib.paged_append(k, v, kp, vp, bad, lens, start, freq=f)
        assert cuda_lib.sync_status() == cuda_lib.FA_ERR_INDEX
    # only position 17 .. 19 and 38, 39 were named, all on bad pages: nothing was written
    assert torch.equal(kp, before[0]) and torch.equal(vp, before[1])
    # a length beyond the table, a negative one, offsets out of order or behind the tokens
    for a in (dict(lens=[20, 1 << 20]), dict(lens=[20, -1]), dict(start=[0, 4, 3]),
              dict(start=[0, 3, 77])):
        n = torch.tensor(a.get("lens", [20, 40]), dtype=torch.int32, device=DEV)
        st = torch.tensor(a.get("start", [0, 3, 5]), dtype=torch.int32, device=DEV)
        kp.copy_(before[0])
        cuda_lib.paged_append(k, v, kp, vp, table, n, st, freq=f)
        assert cuda_lib.sync_status() == cuda_lib.FA_ERR_INDEX, a
        other = torch.ones(kp.shape[0], dtype=torch.bool, device=DEV)
        other[int(t.table[0, 1])] = False  # the good sequence's tokens may be there
        if "lens" in a:  # the bad one wrote nowhere
            assert torch.equal(kp[other], before[0][other])


def test_prompt_then_tokens_equals_one_long_sequence(cuda_lib):
    """Chunks, then single tokens, appended and attended step by step, against the rotation and the
    forward of the whole sequence at once."""
    H, Hkv, d, page, N = 8, 2, 128, 16, 333
    g = torch.Generator().manual_seed(50)
    f, _ = cuda_lib.rope_frequencies(d, device=DEV)
    B = 2
    qkv = torch.randn((B, N, H + 2 * Hkv, d), generator=g).to(BF).to(DEV)
    q, k, v = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
    qr, kr = cuda_lib.rope(q, k, f)
    want, want_lse = cuda_lib.fwd_gqa(qr, kr, v.contiguous(), causal=True)
    pages = -(-N // page)
    kp = torch.full((B * pages, Hkv, page, d), float("nan"), dtype=BF, device=DEV)
    vp = kp.clone()
    table = torch.randperm(B * pages, generator=g).to(torch.int32).view(B, pages).to(DEV)
    got = torch.zeros(B, N, H, d, dtype=BF, device=DEV)
    lse = torch.zeros(B, N, H, device=DEV)
    at = [0, 0]
    for step in [(200, 7), (100, 0), (1, 1), (1, 300), (2, 4), (29, 21)]:
        rows = [list(range(at[b], at[b] + step[b])) for b in range(B)]
        at = [at[b] + step[b] for b in range(B)]
        toks = torch.cat([qkv[b, rows[b]] for b in range(B)])
        lens = torch.tensor(at, dtype=torch.int32, device=DEV)
        start = torch.tensor([0, step[0], sum(step)], dtype=torch.int32, device=DEV)
        x = cuda_lib.paged_append(toks[:, H:H + Hkv], toks[:, H + Hkv:], kp, vp, table, lens, start,
                                  q=toks[:, :H], freq=f)
        o, l = cuda_lib.paged_attention(x, kp, vp, table, lens, start, max_q=max(step))
        for b, (p, n) in enumerate(((0, step[0]), (step[0], step[1]))):
            got[b, rows[b]] = o[p:p + n]
            lse[b, rows[b]] = l[p:p + n]
    assert at == [N, N] and cuda_lib.sync_status() == 0
    # both sides round P and O to bf16 once; their O differ by no more than the sum of the two bounds
    rel = float((got.transpose(1, 2).float() - want.float()).norm() / want.float().norm())
    assert rel <= 2 * 5e-3 and float((lse.transpose(1, 2) - want_lse).abs().max()) <= 2e-3


def test_captured_decode_steps_of_two_layers(cuda_lib):
    """One step (a position more, then append and attention of two layers) captured once and replayed
    token by token gives the eager steps' bits, and these the definition's values."""
    H, Hkv, d, page, steps, lens0 = 6, 2, 64, 16, 5, (12, 300, 0, 127)
    B = len(lens0)
    f, _ = cuda_lib.rope_frequencies(d, device=DEV)
    g = torch.Generator().manual_seed(60)
    x = torch.randn((steps, 2, B, H + 2 * Hkv, d), generator=g).to(HF).to(DEV)
    layers = [Batch([(1, L + steps) for L in lens0], H, Hkv, d, HF, page, seed=61 + i, poison=False)
              for i in range(2)]

    def run(graph):
        caches = [tuple(y.to(DEV) for y in (t.k, t.v, t.table)) for t in layers]
        now = torch.empty_like(x[0])
        lens = torch.tensor(lens0, dtype=torch.int32, device=DEV)
        bufs = [(torch.empty(B, H, d, dtype=HF, device=DEV), torch.empty(B, H, device=DEV),
                 torch.empty(B, H, d, dtype=HF, device=DEV)) for _ in range(2)]

        def step():
            lens.add_(1)
            for (kp, vp, table), (o, l, qr), y in zip(caches, bufs, now):
                q, k, v = y[:, :H], y[:, H:H + Hkv], y[:, H + Hkv:]
                cuda_lib.paged_append(k, v, kp, vp, table, lens, q=q, out_q=qr, freq=f)
                cuda_lib.paged_attention(qr, kp, vp, table, lens, max_q=1, out=o, lse=l)

        if graph:
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
            step = captured.replay
        seen = []
        for i in range(steps):
            now.copy_(x[i])
            step()
            seen += [y.clone() for b in bufs for y in b]
        return seen, caches

    want, caches = run(False)
    got, caches2 = run(True)
    assert cuda_lib.sync_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for t, a, b, at in zip(layers, caches, caches2, (-6, -3)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        t.k, t.v, t.q = a[0].cpu(), a[1].cpu(), want[at + 2].cpu()
        check(t, want[at], want[at + 1], d ** -0.5, True, "last step")


def test_many_sequences(cuda_lib):
    """More sequences than a warp finds in two reads, most of them short, many without a new token."""
    g = torch.Generator().manual_seed(70)
    lens = torch.randint(0, 40, (1500,), generator=g).tolist()
    seqs = [(min(L, i % 4), L) for i, L in enumerate(lens)]
    seqs[700] = (90, 900)
    H, Hkv, d = 4, 2, 64
    t = Batch(seqs, H, Hkv, d, BF, 8, seed=71, pad=(2, 5), poison=False)
    _, kp, vp, table, lens, start = t.dev()
    kv = torch.randn((2, t.T, Hkv, d), generator=g).to(BF)
    cuda_lib.paged_append(kv[0].to(DEV), kv[1].to(DEV), kp, vp, table, lens, start)
    for b, (n, L) in enumerate(seqs):
        for i in range(n):
            p, r = int(t.table[b, (L - n + i) // 8]), (L - n + i) % 8
            t.k[p, :, r], t.v[p, :, r] = kv[0, int(t.start[b]) + i], kv[1, int(t.start[b]) + i]
    assert torch.equal(kp.cpu(), t.k) and torch.equal(vp.cpu(), t.v)
    for causal in (True, False):
        o, lse = attend(cuda_lib, t, causal=causal)
        check(t, o, lse, d ** -0.5, causal, "many")
    assert cuda_lib.sync_status() == 0


@pytest.mark.parametrize("H,Hkv,d,dtype", [(4, 2, 128, BF), (6, 3, 64, HF)])
def test_short_sequences_between_ones_that_see_nothing(cuda_lib, H, Hkv, d, dtype):
    """Units of one to three key tiles and units without any, many to a CTA, in every order."""
    g = torch.Generator().manual_seed(75)
    lens = torch.randint(-150, 300, (400,), generator=g).clamp(min=0).tolist()
    t = Batch([(1 + i % 3, L) for i, L in enumerate(lens)], H, Hkv, d, dtype, 16, seed=76, room=9000)
    for causal in (True, False):
        o, lse = attend(cuda_lib, t, causal=causal)
        assert cuda_lib.sync_status() == 0
        check(t, o, lse, d ** -0.5, causal, "short")
