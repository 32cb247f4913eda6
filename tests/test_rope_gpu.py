"""GPU parity of rotary positions (fa_rope) with the fp64 definition, element by element.

Tolerance, derived: the angle is exact to 2^-33 turns and reaches the sine as a 24-bit float of
half turns (error below 2^-24 pi), sine and cosine are good to 2 units in the last place, and the
two products and their sum round three times in fp32, so before the final rounding a pair's element
is off by less than 2^-20 mscale (|a| + |c|); the rounding to 16 bits adds half a unit, eps / 2
relative to the value (fp16 below 2^-14: half of 2^-24).
"""
import numpy as np
import pytest
import torch

from oracle import paged as op

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def draw(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def near(got, x, ref, rot, interleaved, mscale, what):
    """got: the library's tensor; x its input (CPU), ref the fp64 result."""
    x = x.double().numpy()
    a, c = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    mag = np.zeros_like(x)
    mag[..., a] = mag[..., c] = np.abs(x[..., a]) + np.abs(x[..., c])
    d = 2.0 ** -20 * mscale * mag
    eps = torch.finfo(got.dtype).eps
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= d + eps / 2 * (np.abs(ref) + d) + tiny).all(), what
    assert np.array_equal(got.double().cpu().numpy()[..., rot:], x[..., rot:]), what


CASES = [  # B, H, Hkv, N, d, rot, interleaved, dtype, positions start
    (1, 1, 1, 1, 64, 64, False, torch.bfloat16, None),
    (2, 3, 1, 5, 128, 128, False, torch.float16, 7),
    (1, 6, 2, 33, 64, 16, True, torch.bfloat16, 131072),
    (3, 4, 4, 17, 128, 48, False, torch.float16, 2000000),
    (2, 5, 0, 129, 128, 128, True, torch.float16, None),
    (1, 32, 8, 200, 128, 96, True, torch.bfloat16, -100),
    (2, 7, 7, 61, 64, 48, False, torch.bfloat16, 2147483647 - 61),
]


@pytest.mark.parametrize("B,H,Hkv,N,d,rot,inter,dtype,start", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_parity(cuda_lib, B, H, Hkv, N, d, rot, inter, dtype, start, inverse):
    f = op.inverse_frequencies(rot)
    table, _ = cuda_lib.rope_frequencies(rot, device=DEV)
    q = draw((B, H, N, d), dtype, 1)
    k = draw((B, Hkv, N, d), dtype, 2) if Hkv else None
    pos = np.broadcast_to(np.arange(N), (B, N)) if start is None else \
        start + np.arange(N) + np.zeros((B, 1), dtype=np.int64)
    given = None if start is None else torch.from_numpy(pos.astype(np.int32)).to(DEV)
    call = cuda_lib.rope_bwd if inverse else cuda_lib.rope
    out = call(q.to(DEV), None if k is None else k.to(DEV), table, given, inter, 1.25)
    for x, y in zip((q, k) if Hkv else (q,), out if Hkv else (out,)):
        ref = op.rope(x, pos[:, None, :], f, inter, 1.25, inverse)
        near(y, x, ref, rot, inter, 1.25, "rope")
        assert y.is_contiguous()
    assert cuda_lib.sync_status() == 0


@pytest.mark.parametrize("inter", [False, True])
def test_rope_reads_and_writes_slices_of_a_joint_projection_and_in_place(cuda_lib, inter):
    B, H, Hkv, N, d, rot = 2, 6, 2, 41, 64, 32
    table, _ = cuda_lib.rope_frequencies(rot, device=DEV)
    joint = draw((B, N, H + 2 * Hkv, d), torch.bfloat16, 3)
    dev = joint.to(DEV)
    q, k = dev[:, :, :H].transpose(1, 2), dev[:, :, H:H + Hkv].transpose(1, 2)
    a = cuda_lib.rope(q, k, table, interleaved=inter)
    b = cuda_lib.rope(q.contiguous(), k.contiguous(), table, interleaved=inter)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # written back into a projection's gradient: the slices change, the rest of it does not
    grad = torch.full_like(dev, 7.0)
    gq, gk = grad[:, :, :H].transpose(1, 2), grad[:, :, H:H + Hkv].transpose(1, 2)
    cuda_lib.rope(q, k, table, interleaved=inter, out_q=gq, out_k=gk)
    assert torch.equal(gq, a[0]) and torch.equal(gk, a[1])
    assert bool((grad[:, :, H + Hkv:] == 7.0).all())
    cuda_lib.rope(q, k, table, interleaved=inter, out_q=q, out_k=k)
    assert torch.equal(q, a[0]) and torch.equal(k, a[1])
    assert torch.equal(dev[:, :, H + Hkv:].cpu(), joint[:, :, H + Hkv:])
    # a broadcast input (one head for all) and an expanded batch
    one = draw((1, 1, N, d), torch.bfloat16, 4).to(DEV)
    y = cuda_lib.rope(one.expand(3, 4, N, d), None, table, interleaved=inter)
    z = cuda_lib.rope(one, None, table, interleaved=inter)
    assert all(torch.equal(y[i, j], z[0, 0]) for i in range(3) for j in range(4))


def test_rope_stretched_tables(cuda_lib):
    N, d = 50, 128
    x = draw((1, 2, N, d), torch.float16, 5)
    pos = 60000 + np.arange(N)
    for kind, extra in (("linear", ()), ("ntk", ()), ("by_parts", (8192.0, 1.0, 32.0)),
                        ("bands", (8192.0, 1.0, 4.0))):
        table, m = cuda_lib.rope_frequencies(d, 5e5, kind, 8.0, *extra, device=DEV)
        f = np.array([t % 2 ** 64 for t in table.cpu().tolist()]) * (2 * np.pi / 2.0 ** 64)
        y = cuda_lib.rope(x.to(DEV), None, table, torch.from_numpy(pos.astype(np.int32)[None]).to(DEV),
                          mscale=m)
        near(y, x, op.rope(x, pos[None, None], f, False, m), d, False, m, kind)


def test_rope_then_attention_trains(cuda_lib):
    """Rotation, grouped attention and both backwards in a row against autograd in 64 bits."""
    B, H, Hkv, N, d, rot = 1, 4, 2, 150, 64, 64
    table, _ = cuda_lib.rope_frequencies(rot, device=DEV)
    t = {n: draw((B, h, N, d), torch.bfloat16, 20 + i)
         for i, (n, h) in enumerate((("q", H), ("k", Hkv), ("v", Hkv), ("do", H)))}
    g = {n: x.to(DEV) for n, x in t.items()}
    qr, kr = cuda_lib.rope(g["q"], g["k"], table)
    o, lse = cuda_lib.fwd_gqa(qr, kr, g["v"], causal=True)
    dqr, dkr, dv = cuda_lib.bwd_gqa(qr, kr, g["v"], o, lse, g["do"], causal=True)
    dq, dk = cuda_lib.rope_bwd(dqr, dkr, table)
    assert cuda_lib.sync_status() == 0
    ref = {n: x.double().requires_grad_(n != "do") for n, x in t.items()}
    ang = torch.arange(N).double()[:, None] * torch.from_numpy(op.inverse_frequencies(rot))

    def turn(x):
        a, c = x[..., :rot // 2], x[..., rot // 2:]
        return torch.cat((a * ang.cos() - c * ang.sin(), c * ang.cos() + a * ang.sin()), -1)
    k2 = turn(ref["k"]).repeat_interleave(H // Hkv, 1)
    s = turn(ref["q"]) @ k2.transpose(-1, -2) / d ** 0.5
    s = s.masked_fill(torch.ones(N, N).triu(1).bool(), float("-inf"))
    out = s.softmax(-1) @ ref["v"].repeat_interleave(H // Hkv, 1)
    out.backward(ref["do"])
    for name, x, y in (("o", o, out.detach()), ("dq", dq, ref["q"].grad), ("dk", dk, ref["k"].grad),
                       ("dv", dv, ref["v"].grad)):
        rel = float((x.double().cpu() - y).norm() / y.norm())
        # the attention's own bar is 1e-2 on gradients; each rotation adds one rounding, 2^-9 at most
        assert rel <= (5e-3 if name == "o" else 1e-2) + 2 * 2.0 ** -9, (name, rel)


def test_rope_other_stream_and_graph(cuda_lib):
    table, _ = cuda_lib.rope_frequencies(64, device=DEV)
    q = draw((2, 4, 70, 64), torch.bfloat16, 6).to(DEV)
    want = cuda_lib.rope(q, None, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cuda_lib.rope(q, None, table, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.rope(q, None, table, out_q=out)
    q.copy_(draw((2, 4, 70, 64), torch.bfloat16, 7).to(DEV))
    graph.replay()
    assert torch.equal(out, cuda_lib.rope(q, None, table))


def test_rope_refusals_on_device(cuda_lib):
    table, _ = cuda_lib.rope_frequencies(64, device=DEV)
    q = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(k=q[:1]), dict(k=q.half()), dict(freq=table.cpu()), dict(freq=table.float()),
                dict(positions=torch.zeros(2, 8, device=DEV)), dict(out_q=q[:1]),
                dict(positions=torch.zeros(2, 7, dtype=torch.int32, device=DEV)), dict(out_k=q),
                dict(q=q.transpose(2, 3)[:, :, :8, :4])):
        args = dict(q=q, k=None, freq=table)
        args.update(bad)
        with pytest.raises((ValueError, TypeError)):
            cuda_lib.rope(**args)
    with pytest.raises(TypeError):
        cuda_lib.rope(q.float(), None, table)
    with pytest.raises(cuda_lib.FAError):  # 20 rotated elements: not a multiple of 16
        cuda_lib.rope(q, None, table[:10].contiguous())
    with pytest.raises(cuda_lib.FAError):  # a head stride that is no multiple of 8
        cuda_lib.rope(torch.zeros(2, 4, 8, 68, dtype=torch.bfloat16, device=DEV)[..., :64], None, table)
