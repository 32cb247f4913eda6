"""Rotary positions where a pair's element comes from its partner alone, so that what counts is the
relative error of the sine, not the absolute one that test_rope_gpu allows: most pairs of a row turn
by little over a whole prompt.

Tolerance, derived, for an input of one element c per pair (the other is zero) and angles t of up to
pi / 2: the angle is cut to 2^-32 turns, 2 pi 2^-32 in absolute terms, and then rounded to 24 bits
(2^-24 relative, twice with the product by 2 pi 2^-32); below 1/4 the sine is its series to t^5, off
by t^6 / 5040 < 2^-24 relative and four roundings of 2^-24; from 1/4 on the special-function unit's
2^-21.4 is 2^-19.4 of a sine of at least 0.247.  Two roundings follow (mscale, the product).  All of
it is below 2^-19 relative; the rounding to 16 bits adds eps / 2 (fp16 below 2^-14: 2^-25).

At any angle, sine and cosine from the special-function unit are off by up to 2^-21.2, and the angle's
rounding (2^-24 twice, of up to pi: 2^-22.3) comes on top: together 2^-20.6 of |a| + |c|, with the three
fp32 roundings of a product and a sum (2^-24 each) below 2^-20 (|a| + |c|), the bound of test_rope_gpu.
"""
import numpy as np
import pytest
import torch

from oracle import paged as op

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,rot,base", [(128, 128, 5e5), (64, 64, 1e4), (128, 64, 1e6)])
@pytest.mark.parametrize("inverse", [False, True])
def test_small_angles_keep_their_bits(cuda_lib, interleaved, dtype, d, rot, base, inverse):
    N = 700
    f = op.inverse_frequencies(rot, base)
    table, _ = cuda_lib.rope_frequencies(rot, base, device=DEV)
    a, c = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    call = cuda_lib.rope_bwd if inverse else cuda_lib.rope
    eps, tiny = torch.finfo(dtype).eps, 2.0 ** -25 if dtype == torch.float16 else 0.0
    t = np.arange(N)[:, None] * f
    near = (t <= np.pi / 2) & (t > 0)
    assert near.any(0).sum() > rot // 3  # most pairs, over a good part of the rows
    for filled, other, sign in ((a, c, 1.0), (c, a, -1.0)):
        x = torch.zeros(1, 1, N, d, dtype=dtype)
        x[..., filled] = 1.5
        y = call(x.to(DEV), None, table, interleaved=interleaved, mscale=1.25)
        ref = sign * (-1.0 if inverse else 1.0) * np.sin(t) * 1.25 * 1.5
        err = np.abs(y.double().cpu().numpy()[0, 0][:, other] - ref)
        before = 2 * np.pi * 2.0 ** -32 * 1.25 * 1.5 + 2.0 ** -19 * np.abs(ref)
        bound = before + eps / 2 * (np.abs(ref) + before) + tiny
        worst = (err / bound)[near].max()
        assert worst <= 1, f"off by {worst:.3g} times the bound"
    assert cuda_lib.sync_status() == 0
