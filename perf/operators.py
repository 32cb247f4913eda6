"""Measured cases of the rotary-position and paged-cache operators.

Three operators that a serving or training step with attention calls one after the other:

* ``rope``   rotary positions on Q and K in one call, forward and backward (``api.rope``,
             ``api.rope_bwd``): both pair layouts, part of the head, stretched positions;
* ``append`` the new tokens' K (rotated on the way) and V into a paged cache, Q rotated beside
             them (``api.paged_append``);
* ``attend`` attention of the new tokens of every sequence, one or many, over the paged cache
             (``api.paged_attention``).

``run`` computes them in their plain form, or, where ``own`` is set, calls the library.  ``exact``
computes them from their definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------ cases
def rope_case(name, way, B, H, Hkv, N, d, rot, interleaved, dtype, factor=1.0, start=0):
    c = dict(op="rope", way=way, B=B, H=H, Hkv=Hkv, N=N, d=d, rot=rot, interleaved=interleaved,
             dtype=dtype, factor=factor, start=start)
    return dict(c, name=name) if name else c


def append_case(name, B, chunks, n, ctx, H, Hkv, d, page, rot, interleaved, dtype, token_rows,
                factor=1.0):
    c = dict(op="append", B=B, chunks=chunks, n=n, ctx=ctx, H=H, Hkv=Hkv, d=d, page=page, rot=rot,
             interleaved=interleaved, dtype=dtype, token_rows=token_rows, factor=factor)
    return dict(c, name=name) if name else c


def attend_case(name, B, chunks, n, ctx, ragged, H, Hkv, d, page, dtype, token_rows):
    c = dict(op="attend", B=B, chunks=chunks, n=n, ctx=ctx, ragged=ragged, H=H, Hkv=Hkv, d=d,
             page=page, dtype=dtype, token_rows=token_rows)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short prompt of a small model, half of each head rotated, adjacent pairs
        rope_case("rope_small", "fwd", 2, 6, 2, 37, 64, 32, True, "fp16"),
        # the 8k training shape with grouped heads, Q and K read out of the joint projection
        rope_case("rope_fwd_n8k", "fwd", 1, 32, 8, 8192, 128, 128, False, "bf16"),
        # the gradients of the 4k training shape, written back in the projection's layout
        rope_case("rope_bwd_n4k", "bwd", 2, 16, 16, 4096, 128, 128, False, "bf16"),
        # a long-context fine-tune's gradient: far positions squeezed by 4, odd length
        rope_case("rope_bwd_far_n1023", "bwd", 4, 16, 16, 1023, 64, 32, True, "fp16", 4.0, 131072),
        # one generated token for each of 16 sequences
        append_case("append_decode", 16, 0, 1, 1024, 32, 8, 128, 16, 128, False, "bf16", False),
        # prompt chunks of six sequences
        append_case("append_chunks", 6, 6, 2048, 1500, 32, 8, 128, 64, 128, False, "bf16", False),
        # two prompts beside three generating sequences, token rows outside heads in the pages
        append_case("append_mixed_d64", 5, 2, 300, 700, 12, 4, 64, 32, 32, True, "fp16", True, 2.0),
        # one sequence generating a token after a short prompt: nothing but latency
        attend_case("attend_one", 1, 0, 1, 1000, False, 32, 8, 128, 16, "bf16", False),
        # one token for each of 16 sequences over 8k cached keys
        attend_case("attend_decode_8k", 16, 0, 1, 8191, False, 32, 8, 128, 16, "bf16", False),
        # four drafted tokens each to be verified at once, ragged caches, small heads
        attend_case("attend_verify_d64", 8, 8, 4, 4096, True, 16, 2, 64, 64, "fp16", True),
        # two prompt chunks in the batch of 18 generating sequences
        attend_case("attend_mixed", 20, 2, 500, 2500, True, 32, 8, 128, 32, "bf16", False),
        # the last quarter of an 8k prompt over the three quarters already cached
        attend_case("attend_chunk_8k", 1, 1, 2048, 6144, False, 32, 8, 128, 128, "bf16", False),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["rope", "append", "attend"])
    dtype = rng.choice(["bf16", "fp16"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    rep = rng.choice([1, 2, 3, 4, 7, 8])
    H = min(Hkv * rep, 32 // Hkv * Hkv)
    rot = rng.choice([d, d, d // 2, d // 4])
    inter = rng.random() < 0.5
    page = rng.choice([16, 32, 64, 128, 256])
    rows = rng.random() < 0.3
    factor = rng.choice([1.0, 1.0, 4.0])
    if op == "rope":
        B = rng.choice([1, 2, 4])
        return rope_case(None, rng.choice(["fwd", "bwd"]), B, H, Hkv, log(5, 8192 // B), d, rot,
                         inter, dtype, factor, rng.choice([0, 0, 9000, 200000]))
    if op == "append":
        B = log(1, 32)
        chunks = rng.choice([0, B // 4, B])
        n = log(2, 8192 // max(B, 8)) if chunks else 1
        return append_case(None, B, chunks, n, log(16, 1500), H, Hkv, d, page, rot, inter, dtype,
                           rows, factor)
    if rng.random() < 0.5:  # generating sequences, or a few drafted tokens each
        B = log(1, 32)
        few = rng.choice([1, 1, 2, 5])
        return attend_case(None, B, B if few > 1 else 0, few, log(20, 65536 // max(B, 8)),
                           rng.random() < 0.7, H, Hkv, d, page, dtype, rows)
    B = rng.choice([1, 2, 5, 12])  # prompt chunks, alone or among generating sequences
    chunks = 1 if B < 5 else 2
    return attend_case(None, B, chunks, log(30, 1400 // chunks), log(30, 5000), B > 1, H, Hkv, d, page,
                       dtype, rows)


def lengths(c):
    """New tokens and cached tokens before them of each sequence: part of the case's sizes."""
    r = random.Random(c["B"] * 7919 + c["n"] * 31 + c["ctx"])
    ragged = c.get("ragged", True)
    new, ctx = [], []
    for b in range(c["B"]):
        chunk = b < c["chunks"]
        n = c["n"] if chunk else 1
        if chunk and ragged and c["n"] > 8:
            n = r.randint(c["n"] // 2, c["n"])
        new.append(n)
        ctx.append(r.randint(c["ctx"] // 2, c["ctx"]) if ragged else c["ctx"])
    order = list(range(c["B"]))
    r.shuffle(order)
    return [new[i] for i in order], [ctx[i] for i in order]


# ------------------------------------------------------------------------------------------ inputs
def inverse_frequencies(c):
    """Radians per position of each pair, in 64 bits; `factor` squeezes the positions."""
    i = np.arange(c["rot"] // 2, dtype=np.float64)
    return 10000.0 ** (-2.0 * i / c["rot"]) / c["factor"]


def frequency_table(c):
    """The same as turns per position in units of 2^-64 turns, which a program keeps."""
    turns = inverse_frequencies(c) / (2.0 * math.pi)
    return torch.tensor([int(math.ldexp(t, 64)) for t in turns], dtype=torch.int64).to(DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = random.Random(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(t)

    s = dict(case=c)
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    if c["op"] != "attend":
        s["inv_freq"] = torch.from_numpy(inverse_frequencies(c)).to(DEV)
        s["freq"] = frequency_table(c)
    if c["op"] == "rope":
        B, N = c["B"], c["N"]
        base = torch.tensor([[c["start"] + host.randrange(1000)] for _ in range(B)])
        s["positions"] = (base + torch.arange(N)[None, :]).to(torch.int32).to(DEV)
        joint = normal(B, N, H + 2 * Hkv, d)  # the joint projection of Q, K and V
        if c["way"] == "fwd":
            s["q"] = joint[:, :, :H].transpose(1, 2)
            s["k"] = joint[:, :, H:H + Hkv].transpose(1, 2)
        else:
            s["dq"], s["dk"] = normal(B, H, N, d), normal(B, Hkv, N, d)
            s["out_q"] = joint[:, :, :H].transpose(1, 2)
            s["out_k"] = joint[:, :, H:H + Hkv].transpose(1, 2)
        return s
    new, ctx = lengths(c)
    B, page = c["B"], c["page"]
    total = sum(new)
    kv_len = [a + b for a, b in zip(new, ctx)]
    pages = [-(-x // page) for x in kv_len]
    width, pool = max(pages), sum(pages) + 3
    ids = list(range(pool))
    host.shuffle(ids)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = torch.tensor(ids[at:at + pages[b]], dtype=torch.int32)
        at += pages[b]
    s["table"] = table.to(DEV)
    s["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    s["q_start"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
    s["max_q"], s["max_kv"] = max(new), max(kv_len)  # a scheduler knows them
    if c["token_rows"]:  # a token's heads side by side within a page
        s["k_pages"] = normal(pool, page, Hkv, d).transpose(1, 2)
        s["v_pages"] = normal(pool, page, Hkv, d).transpose(1, 2)
    else:
        s["k_pages"], s["v_pages"] = normal(pool, Hkv, page, d), normal(pool, Hkv, page, d)
    if c["op"] == "append":
        joint = normal(total, H + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = joint[:, :H], joint[:, H:H + Hkv], joint[:, H + Hkv:]
    else:
        s["q"] = normal(total, H, d)
    return s


# ------------------------------------------------------------------------------------- plain forms
def plain_rotate(x, angle, rot, interleaved):
    """x [..., d] rotated by angle [..., rot / 2] (64 bits), in 32 bits."""
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    f = x.float()
    head, rest = f[..., :rot], f[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        out = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        out = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((out, rest), dim=-1).to(x.dtype)


def plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, :, None] * s["inv_freq"]
    if c["way"] == "fwd":
        return [plain_rotate(s[n], angle, c["rot"], c["interleaved"]).contiguous() for n in "qk"]
    s["out_q"].copy_(plain_rotate(s["dq"], -angle, c["rot"], c["interleaved"]))
    s["out_k"].copy_(plain_rotate(s["dk"], -angle, c["rot"], c["interleaved"]))
    return [s["out_q"], s["out_k"]]


def token_places(s):
    """Sequence and place within it of every token."""
    total = s["q"].shape[0]
    tok = torch.arange(total, device=DEV)
    seq = torch.searchsorted(s["q_start"].long(), tok, right=True) - 1
    return seq, tok - s["q_start"].long()[seq]


def plain_append(s):
    c = s["case"]
    seq, place = token_places(s)
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    pos = s["kv_len"].long()[seq] - n[seq] + place
    angle = pos.double()[:, None, None] * s["inv_freq"]
    q = plain_rotate(s["q"], angle, c["rot"], c["interleaved"]).contiguous()
    page = s["table"].long()[seq, pos // c["page"]]
    row = pos % c["page"]
    s["k_pages"][page, :, row] = plain_rotate(s["k"], angle, c["rot"], c["interleaved"])
    s["v_pages"][page, :, row] = s["v"]
    return [q, s["k_pages"], s["v_pages"]]


def plain_attend(s):
    c = s["case"]
    B, H, Hkv, d, page = c["B"], c["H"], c["Hkv"], c["d"], c["page"]
    rep, nq, L = H // Hkv, s["max_q"], s["max_kv"]
    first = s["q_start"][:-1].long()
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    kv_len = s["kv_len"].long()
    # every sequence's queries and keys, padded to the longest
    tok = (first[:, None] + torch.arange(nq, device=DEV)).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][tok].float().view(B, nq, Hkv, rep, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, rep * nq, d)
    pos = torch.arange(L, device=DEV)
    ids = s["table"].long()[:, pos // page].clamp(min=0)
    row = (pos % page).expand(B, L)
    there = pos < kv_len[:, None]
    k = s["k_pages"][ids, :, row].float().permute(0, 2, 1, 3)
    v = s["v_pages"][ids, :, row].float().permute(0, 2, 1, 3)
    v = torch.where(there[:, None, :, None], v, torch.zeros((), device=DEV))
    score = (torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))).view(B, Hkv, rep, nq, L)
    last = (kv_len - n)[:, None] + torch.arange(nq, device=DEV)
    seen = pos <= last[:, :, None]
    score = score.masked_fill(~(seen & there[:, None])[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, rep * nq, L), v).view(B, Hkv, rep, nq, d)
    o = o / torch.where(total > 0, total, torch.ones((), device=DEV))
    lse = (top + torch.log(total)).squeeze(-1)
    seq, place = token_places(s)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, nq, H, d)[seq, place]
    return [o.to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(B, nq, H)[seq, place]]


def own_run(s):
    from exact_attention_staged_gb300 import api
    c = s["case"]
    if c["op"] == "rope" and c["way"] == "fwd":
        return list(api.rope(s["q"], s["k"], s["freq"], positions=s["positions"],
                             interleaved=c["interleaved"]))
    if c["op"] == "rope":
        return list(api.rope_bwd(s["dq"], s["dk"], s["freq"], positions=s["positions"],
                                 interleaved=c["interleaved"], out_q=s["out_q"], out_k=s["out_k"]))
    if c["op"] == "append":
        q = api.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["kv_len"],
                             q_start=s["q_start"], q=s["q"], freq=s["freq"],
                             interleaved=c["interleaved"])
        return [q, s["k_pages"], s["v_pages"]]
    return list(api.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_len"],
                                    q_start=s["q_start"], max_q=s["max_q"], causal=True))


def run(state):
    if own:
        return own_run(state)
    return {"rope": plain_rope, "append": plain_append, "attend": plain_attend}[state["case"]["op"]](state)


# -------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    if c["op"] == "rope":
        rows = c["B"] * c["N"]
        return {"bytes": 2 * rows * (H + Hkv) * d * 2 + 4 * rows + 4 * c["rot"],
                "flops": 3 * rows * (H + Hkv) * c["rot"]}
    new, ctx = lengths(c)
    total, tables = sum(new), sum(-(-(a + b) // c["page"]) for a, b in zip(new, ctx))
    small = 8 * c["B"] + 4
    if c["op"] == "append":
        touched = sum((a + b - 1) // c["page"] - b // c["page"] + 1 for a, b in zip(new, ctx))
        return {"bytes": 2 * total * (H + 2 * Hkv) * d * 2 + 4 * touched + small + 4 * c["rot"],
                "flops": 3 * total * (H + Hkv) * c["rot"]}
    keys = sum(new) + sum(ctx)
    seen = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, ctx))
    return {"bytes": keys * Hkv * d * 4 + total * H * d * 4 + total * H * 4 + 4 * tables + small,
            "flops": 4 * seen * H * d}


# --------------------------------------------------------------------------- definitions in 64 bits
def exact_pairs(x, pos, inv_freq, rot, interleaved, sign):
    """Each pair as a complex number times e^(i sign pos inv_freq); x [rows, heads, d], pos [rows]."""
    f = x.double()
    out = f.clone()
    at = torch.arange(rot // 2, device=x.device)
    first, second = (2 * at, 2 * at + 1) if interleaved else (at, at + rot // 2)
    z = torch.complex(f[..., first], f[..., second])
    turn = torch.polar(torch.ones_like(inv_freq)[None, :].expand(len(pos), -1),
                       sign * pos.double()[:, None] * inv_freq[None, :])
    z = z * turn[:, None, :]
    out[..., first] = z.real
    out[..., second] = z.imag
    return out


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    if c["op"] == "rope":
        sign = 1.0 if c["way"] == "fwd" else -1.0
        outs = []
        for x in ((s["q"], s["k"]) if c["way"] == "fwd" else (s["dq"], s["dk"])):
            rows = x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], d)
            y = exact_pairs(rows, s["positions"].reshape(-1), s["inv_freq"], c["rot"],
                            c["interleaved"], sign)
            outs.append(y.view(c["B"], c["N"], x.shape[1], d).transpose(1, 2))
        return outs
    new, ctx = lengths(c)
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    if c["op"] == "append":
        outs = [[], s["k_pages"].double(), s["v_pages"].double()]
        table = s["table"].cpu()
        for b in range(c["B"]):
            pos = torch.arange(ctx[b], ctx[b] + new[b])
            mine = slice(starts[b], starts[b + 1])
            ids = table[b][pos // c["page"]].long().to(DEV)
            rows = (pos % c["page"]).to(DEV)
            pos = pos.to(DEV)
            outs[0].append(exact_pairs(s["q"][mine], pos, s["inv_freq"], c["rot"], c["interleaved"], 1.0))
            outs[1][ids, :, rows] = exact_pairs(s["k"][mine], pos, s["inv_freq"], c["rot"],
                                                c["interleaved"], 1.0)
            outs[2][ids, :, rows] = s["v"][mine].double()
        return [torch.cat(outs[0])] + outs[1:]
    rep = H // Hkv
    o = torch.zeros(sum(new), H, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(sum(new), H, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        L = new[b] + ctx[b]
        ids = s["table"][b, :-(-L // c["page"])].long()
        last = torch.arange(ctx[b], L, device=DEV)
        hidden = torch.arange(L, device=DEV)[None, :] > last[:, None]
        for kh in range(Hkv):
            k = s["k_pages"][ids, kh].reshape(-1, d)[:L].double()
            v = s["v_pages"][ids, kh].reshape(-1, d)[:L].double()
            for h in range(kh * rep, (kh + 1) * rep):
                x = (s["q"][starts[b]:starts[b + 1], h].double() @ k.T) / math.sqrt(d)
                x.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(x, dim=1)
                lse[starts[b]:starts[b + 1], h] = z
                o[starts[b]:starts[b + 1], h] = torch.exp(x - z[:, None]) @ v
    return [o, lse]
