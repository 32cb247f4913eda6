"""Paged cache: what the bounds of a call, its index arrays and values that are not finite may and may
not change.  Attention is compared with the fp64 definition under the bounds that test_paged_gpu
derives; what has to be left alone, or is promised exactly, is compared bit by bit."""
import copy

import pytest
import torch

from test_paged_gpu import BF, DEV, HF, Batch, attend, check

pytestmark = pytest.mark.gpu


# tokens beyond max_q are left out; those before them stay where they stand in the sequence
@pytest.mark.parametrize("room", [0, 9000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("seqs,max_q,H,Hkv,d,dtype", [
    ([(5, 50), (1, 300)], 2, 4, 2, 64, BF),
    ([(2, 129), (4, 130), (3, 700)], 1, 8, 2, 128, HF),
    ([(40, 1000), (9, 20)], 30, 6, 2, 64, HF),
    ([(300, 700), (5, 64), (1, 90)], 140, 4, 2, 128, BF),
    ([(20, 12), (3, 2000)], 11, 4, 1, 64, BF),  # some of the first tokens see nothing
])
def test_tokens_beyond_max_q_leave_the_others_right(cuda_lib, seqs, max_q, H, Hkv, d, dtype, causal, room):
    t = Batch(seqs, H, Hkv, d, dtype, 16, seed=80 + max_q, room=room)
    out = torch.full((t.T, H, d), 3.0, dtype=dtype, device=DEV)
    lse = torch.full((t.T, H), 3.0, device=DEV)
    attend(cuda_lib, t, causal=causal, max_q=max_q, out=out, lse=lse)
    assert cuda_lib.sync_status() == cuda_lib.FA_ERR_INDEX
    kept = copy.copy(t)
    kept.seqs = [(min(n, max_q), L - n + min(n, max_q) if causal else L) for n, L in seqs]
    if causal:  # (a sequence that ends before its kept tokens: they see nothing, checked below)
        kept.seqs = [(n, L) if L > 0 else (0, 0) for n, L in kept.seqs]
    check(kept, out, lse, d ** -0.5, causal, "kept")
    for b, (n, L) in enumerate(seqs):
        at = int(t.start[b])
        if causal and L - n < 0:
            none = slice(at, at + min(n - L, max_q))
            assert bool((out[none] == 0).all()) and bool(torch.isneginf(lse[none]).all())
        left = slice(at + min(n, max_q), at + n)
        assert bool((out[left] == 3.0).all()) and bool((lse[left] == 3.0).all())


@pytest.mark.parametrize("room", [0, 9000])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("seqs,H,Hkv,d,dtype", [
    ([(6, 3), (1, 50)], 4, 2, 64, BF),
    ([(150, 20), (2, 1)], 4, 1, 128, HF),
    ([(300, 290), (1, 40)], 4, 2, 128, BF),
    ([(1, 700)] * 200 + [(5, 2)] * 30, 2, 1, 64, BF),
])
def test_rows_that_see_nothing_are_zero_whatever_others_see(cuda_lib, seqs, H, Hkv, d, dtype, value, room):
    t = Batch(seqs, H, Hkv, d, dtype, 16, seed=90, room=room)
    for b, (n, L) in enumerate(seqs):  # the values that the later rows of such a sequence see
        if L < n:
            for pos in range(L):
                t.v[int(t.table[b, pos // 16]), :, pos % 16] = value
    out, lse = attend(cuda_lib, t)
    assert cuda_lib.sync_status() == 0
    for b, (n, L) in enumerate(seqs):
        if L < n:
            rows = slice(int(t.start[b]), int(t.start[b]) + n - L)
            assert bool((out[rows] == 0).all()), f"sequence {b}"
            assert bool(torch.isneginf(lse[rows]).all()), f"sequence {b}"


def test_a_bad_index_does_not_hide_a_wait_that_ran_out(cuda_lib):
    t = Batch([(1, 300), (2, 500)], 4, 2, 64, BF, 16, seed=17, poison=False)
    q, k, v, table, lens, start = t.dev()
    bad = table.clone()
    bad[0, 18] = -1  # of position 299, to which the first sequence's token goes
    new = torch.zeros(t.T, 2, 64, dtype=BF, device=DEV)
    try:
        cuda_lib.debug_set_wait_limit_ns(20_000_000)
        cuda_lib.debug_set_fault(4)
        cuda_lib.paged_attention(q, k, v, table, lens, start, max_q=2)
        cuda_lib.paged_append(new, new, k, v, bad, lens, start)
        assert cuda_lib.sync_status() == cuda_lib.FA_ERR_TIMEOUT
    finally:
        cuda_lib.debug_set_fault(0)
        cuda_lib.debug_set_wait_limit_ns(0)
    cuda_lib.paged_append(new, new, k, v, bad, lens, start)
    assert cuda_lib.sync_status() == cuda_lib.FA_ERR_INDEX
    cuda_lib.paged_append(new, new, k, v, table, lens, start)
    assert cuda_lib.sync_status() == 0


@pytest.mark.parametrize("lens,start", [([20, 1 << 20, 40], [0, 3, 3, 5]), ([20, -7, 40], [0, 3, 3, 5]),
                                        ([20, 30, 1 << 30], [0, 3, 5, 5]), ([20, 30, 40], [5, 3, 3, 3]),
                                        ([20, 30, 40], [9, 9, 9, 9]), ([20, 30, 40], [5, 5, 5, 4])])
def test_append_reports_bad_entries_of_sequences_without_a_token(cuda_lib, lens, start):
    t = Batch([(3, 20), (0, 30), (2, 40)], 4, 2, 64, BF, 16, seed=41, poison=False)
    _, k, v, table, _, _ = t.dev()
    new = torch.zeros(5, 2, 64, dtype=BF, device=DEV)
    cuda_lib.paged_append(new, new, k, v, table, torch.tensor(lens, dtype=torch.int32, device=DEV),
                          torch.tensor(start, dtype=torch.int32, device=DEV))
    assert cuda_lib.sync_status() == cuda_lib.FA_ERR_INDEX


def test_append_reports_the_last_of_many_sequences(cuda_lib):
    # one token, more sequences than the threads of a block, the last one's length out of range
    B = 3000
    k, v = (torch.zeros(4, 2, 16, 64, dtype=BF, device=DEV) for _ in range(2))
    table = torch.zeros(B, 1, dtype=torch.int32, device=DEV)
    lens = torch.ones(B, dtype=torch.int32, device=DEV)
    start = torch.ones(B + 1, dtype=torch.int32, device=DEV)
    start[0] = 0
    new = torch.ones(1, 2, 64, dtype=BF, device=DEV)
    cuda_lib.paged_append(new, new, k, v, table, lens, start)
    assert cuda_lib.sync_status() == 0
    assert bool((k[0, :, 0] == 1).all()) and float(k.float().sum()) == 2 * 64
    lens[-1] = 17
    cuda_lib.paged_append(new, new, k, v, table, lens, start)
    assert cuda_lib.sync_status() == cuda_lib.FA_ERR_INDEX


@pytest.mark.parametrize("what", [dict(lens=[20, 1 << 20, 9]), dict(lens=[20, -1, 9]),
                                  dict(lens=[49, 40, 9]), dict(page=(1, 2, -1)), dict(page=(1, 2, 9)),
                                  dict(page=(0, 1, 1 << 30)), dict(start=[0, 3, 5, 77]),
                                  dict(start=[-2, 3, 5, 6])])
@pytest.mark.parametrize("H", [0, 4])
def test_append_to_bad_sequences_changes_nothing_and_to_good_ones_all(cuda_lib, what, H):
    """Both pools, bit by bit, against pools built from the good sequences' tokens alone."""
    seqs = [(3, 20), (2, 40), (1, 9)]
    t = Batch(seqs, 4, 2, 64, HF, 16, seed=42, poison=False)
    g = torch.Generator().manual_seed(43)
    q, k, v = (torch.randn((6, h, 64), generator=g).to(HF) for h in (4, 2, 2))
    lens, start, table = [L for _, L in seqs], [0, 3, 5, 6], t.table[:, :3].clone()
    lens, start = what.get("lens", lens), what.get("start", start)
    cap, pool = 3 * 16, t.k.shape[0]
    if "page" in what:
        b, i, entry = what["page"]
        table[b, i] = pool if entry == 9 else entry
    want_k, want_v = t.k.clone(), t.v.clone()
    for b in range(3):
        first, end = start[b], start[b + 1]
        if not (0 <= first <= end <= 6 and 0 <= lens[b] <= cap):
            continue
        for tok in range(first, end):
            pos = lens[b] - (end - tok)
            page = int(table[b, pos // 16])
            if 0 <= page < pool:
                want_k[page, :, pos % 16], want_v[page, :, pos % 16] = k[tok], v[tok]
    kp, vp = t.k.to(DEV), t.v.to(DEV)
    got = cuda_lib.paged_append(k.to(DEV), v.to(DEV), kp, vp, table.to(DEV),
                                torch.tensor(lens, dtype=torch.int32, device=DEV),
                                torch.tensor(start, dtype=torch.int32, device=DEV),
                                q=q.to(DEV) if H else None)
    assert cuda_lib.sync_status() == cuda_lib.FA_ERR_INDEX
    assert torch.equal(kp.cpu(), want_k) and torch.equal(vp.cpu(), want_v)
    if H:  # without a rotation Q is copied, that of bad sequences too (the last token of
        # start [.., 77] and the first of [-2, ..] belong to clamped ranges)
        assert torch.equal(got.cpu(), q)


@pytest.mark.parametrize("room", [0, 9000])
def test_sequences_that_share_their_pages(cuda_lib, room):
    t = Batch([(2, 50)] * 3, 4, 2, 64, BF, 16, seed=8, room=room)
    t.table[1:] = t.table[0]
    t.q[2:] = t.q[:2].repeat(2, 1, 1)
    out, lse = attend(cuda_lib, t)
    assert cuda_lib.sync_status() == 0
    check(t, out, lse, 64 ** -0.5, True, "shared")
