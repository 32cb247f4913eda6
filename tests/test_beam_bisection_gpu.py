"""Beam selection where the K-th largest logit of a piece has to be found by bisection: more logits than there is
room for (512) are above the bound even after it was raised twice.

The first bound is the K-th largest maximum of groups of a block's threads.  Here all logits of K - 1 groups are
raised above the others, so that the bound is one of the others' and lets all raised logits through, some 16000 to
32000 of a piece.  Raising it by the K-th largest of 256 pairs of those that were kept leaves 1 - sqrt(1 - K / 256)
of them, for K = 128 0.29 each time: more than 1200 after two, whatever the order in which they were found.

The order is that of one beam's logits, so it is exact; scores are held to the bound derived in test_beam_gpu.py.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DL = 4.2e-6
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def rows(seed, n, V, K, dtype, vec, step):
    """n rows of V logits, those of K - 1 groups of 256 threads (vec side by side to a thread) between 16 and 32, in
    multiples of step (0: any)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    groups = 32 if K <= 16 else 64 if K <= 32 else 128 if K <= 64 else 256
    thread = torch.arange(V, device=DEV) // vec % 256
    high = 16 + 16 * torch.rand(n, V, generator=g, device=DEV)
    if step:
        high = (high / step).floor() * step
    low = torch.randn(n, V, generator=g, device=DEV)
    return torch.where(thread // (256 // groups) < K - 1, high, low).to(dtype)


def best(x, K):
    """Tokens and logarithms of probabilities of each row's K largest, equal ones by place."""
    at = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :K]
    y = x.double()
    return at, torch.gather(y, -1, at) - torch.logsumexp(y, -1, keepdim=True)


def same(api, got, at, s):
    assert api.sync_status() == 0
    assert torch.equal(got[2].long(), at)
    assert bool(((got[0].double() - s).abs() <= DL + 2.0 ** -24 * s.abs()).all())


# logits of which none, a few and hundreds are equal (there are 128 bf16 numbers between 16 and 32)
@pytest.mark.parametrize("dtype,step", [(F32, 0), (F32, 2.0 ** -6), (F32, 4.0), (BF, 0), (HF, 0)])
@pytest.mark.parametrize("odd", [False, True])
def test_pieces_of_a_grid(cuda_lib, odd, dtype, step):
    """320 rows: a piece is a whole row, and rows that start anywhere are read one logit at a time."""
    V = 65535 if odd else 65536
    vec = 1 if odd else 128 // torch.finfo(dtype).bits
    for K in (128, 100, 64, 17):
        x = rows(K, 320, V, K, dtype, vec, step)
        scores = -torch.rand(320, 1, generator=torch.Generator(device=DEV).manual_seed(K), device=DEV)
        assert cuda_lib.beam_select_workspace_bytes(320, 1, V, K) > 0
        got = cuda_lib.beam_select(x[:, None], scores, k=K)
        at, s = best(x, K)
        same(cuda_lib, got, at, scores + s)
        assert torch.equal(got[1].long(), torch.arange(320, device=DEV)[:, None].expand(320, K))


@pytest.mark.parametrize("dtype,step", [(F32, 0), (F32, 2.0 ** -6), (F32, 4.0), (BF, 0), (HF, 0)])
def test_pieces_of_a_cluster(cuda_lib, dtype, step):
    """One request of 16 beams in one launch, of which one is far ahead of the others."""
    V, K, W = 32768, 128, 16
    x = rows(1, W, V, K, dtype, 128 // torch.finfo(dtype).bits, step)
    at, s = best(x, K)
    assert cuda_lib.beam_select_workspace_bytes(1, W, V, K) == 0
    for w in (0, 7, 15):
        scores = torch.full((1, W), -1e4, device=DEV)
        scores[0, w] = 0.0
        got = cuda_lib.beam_select(x[None], scores, k=K)
        same(cuda_lib, got, at[w:w + 1], s[w:w + 1])
        assert bool((got[1] == w).all())


def test_rows_that_mostly_hold_their_highest_value(cuda_lib):
    """Thousands of equals above the bound, and fewer than K numbers above those, found wherever they stand."""
    V, K = 65536, 128
    x = rows(3, 320, V, K, F32, 4, 0)
    x = torch.where(x > 24, torch.full_like(x, 24.0), x)
    g = torch.Generator(device=DEV).manual_seed(4)
    for some in (0, 1, 100, 127):
        y = x.clone()
        where = torch.rand(320, V, generator=g, device=DEV).argsort(-1)[:, :some]
        y.scatter_(1, where, 25 + torch.rand(320, some, generator=g, device=DEV))
        got = cuda_lib.beam_select(y[:, None], torch.zeros(320, 1, device=DEV), k=K)
        at, s = best(y, K)
        same(cuda_lib, got, at, s)
