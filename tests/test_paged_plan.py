"""The plan of paged attention on the CPU where a call bounds the new tokens by max_q."""
import numpy as np
import pytest
import torch

from exact_attention_staged_gb300 import api, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("tiles", [1, 2])
@pytest.mark.parametrize("seqs,max_q", [([(5, 129)], 2), ([(5, 50), (9, 600), (1, 257)], 1),
                                        ([(700, 900), (3, 384), (40, 12)], 300), ([(64, 20)], 50)])
def test_tokens_beyond_max_q_do_not_move_the_others(lib, seqs, max_q, tiles, causal):
    """Each unit's key tiles are those that its last kept token sees from where it stands."""
    tile, Hkv = 16, 2
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
    start = torch.tensor(np.cumsum([0] + [n for n, _ in seqs]), dtype=torch.int32)
    out = np.zeros((4000, 9), dtype=np.int32)
    n = lib.fa_debug_paged_pieces(lens.data_ptr(), start.data_ptr(), int(start[-1]), len(seqs), Hkv, 16,
                                  100, max_q, tile, tiles, causal, 7, out.ctypes.data, len(out))
    want = {}
    for b, (new, L) in enumerate(seqs):
        kept = min(new, max_q)
        for i in range(0, kept, tile * tiles):
            toks = min(tile * tiles, kept - i)
            keys = L - new + i + toks if causal else L
            for g in range(Hkv):
                want[(b, g, int(start[b]) + i, toks)] = max(1, -(-keys // 128))
    got = {}
    for x in out[:n].tolist():
        got[tuple(x[1:5])] = x[7]
    assert got == want


def test_check_of_a_batch_whose_offsets_end_at_or_below_zero(lib):
    table = torch.tensor([[0], [1]], dtype=torch.int32)
    lens = torch.tensor([3, 4], dtype=torch.int32)

    def ok(*start, **kw):
        return api.paged_check(table, lens, torch.tensor(start, dtype=torch.int32), 2, 16, **kw)
    assert ok(0, 0, 0)          # no sequence brings a token
    assert not ok(0, 0, -3)     # offsets below zero are found, not refused
    assert not ok(-1, 0, 0)
    assert not ok(0, -2, -2)
    assert not ok(-4, -4, -4)
    assert ok(0, 1, 3, max_q=2)
