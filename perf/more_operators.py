"""Measured cases of decoding with branches over the paged cache: what picks the continuations of a
step and what keeps the cache's pages.

* ``select``  beam search's selection: the K best continuations over all beams and the whole
              vocabulary from a step's logits (``api.beam_select``); its parents are what the next
              one takes;
* ``branch``  a step of sequences that share pages: what the last step branched off is given back
              (``api.paged_free``), rows of the table are forked to their parents'
              (``api.paged_fork``), the new tokens get pages of their own (``api.paged_reserve``) and
              the shared, partly filled ones are copied in all layers (``api.paged_copy``);
* ``copy``    page copies alone;
* ``compact`` half of the sequences make room (``api.paged_free``), the live pages move to the front
              of the pool (``api.paged_compact``, ``api.paged_copy``) and the sequences come back
              (``api.paged_reserve``), the two halves taking turns.

``run`` computes them in their plain form, or, where ``own`` is set, calls the library.  ``exact``
computes them from their definitions, numbers in 64 bits and tables one entry at a time.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def select_case(name, B, W, V, K, dtype, finished=0.0, masked=0.0):
    """finished: share of beams that have ended; masked: share of tokens that may not follow."""
    c = dict(op="select", B=B, W=W, V=V, K=K, dtype=dtype, finished=finished, masked=masked)
    return dict(c, name=name) if name else c


def copy_case(name, n, tails, L, Hkv, d, page, dtype, token_rows):
    c = dict(op="copy", n=n, tails=tails, L=L, Hkv=Hkv, d=d, page=page, dtype=dtype, token_rows=token_rows)
    return dict(c, name=name) if name else c


def branch_case(name, G, W, ctx, n, L, Hkv, d, page, dtype, token_rows):
    """G sequences branch into W each, with n new tokens in every branch."""
    c = dict(op="branch", G=G, W=W, ctx=ctx, n=n, L=L, Hkv=Hkv, d=d, page=page, dtype=dtype,
             token_rows=token_rows)
    return dict(c, name=name) if name else c


def compact_case(name, B, ctx, L, Hkv, d, page, dtype, token_rows):
    c = dict(op="compact", B=B, ctx=ctx, L=L, Hkv=Hkv, d=d, page=page, dtype=dtype, token_rows=token_rows)
    return dict(c, name=name) if name else c


def listed():
    return [
        # three beams over a small vocabulary of odd size: nothing but latency
        select_case("select_small", 1, 3, 997, 3, "fp32"),
        # one request's four beams over a large vocabulary
        select_case("select_one_128k", 1, 4, 131072, 4, "bf16"),
        # a batch of requests, twice as many candidates as beams
        select_case("select_128k", 64, 4, 131072, 8, "bf16"),
        # a vocabulary of odd size, so that rows start anywhere; beams that have ended, a grammar that
        # rules tokens out
        select_case("select_odd", 16, 5, 50001, 10, "fp16", 0.2, 0.5),
        # wide beams, 32-bit logits
        select_case("select_wide_fp32", 8, 32, 65536, 64, "fp32"),
        # whole pages of every layer (a prefix duplicated for another tenant)
        copy_case("copy_layers", 256, False, 32, 8, 128, 16, "bf16", False),
        # the filled rows of a few pages, token rows outside heads in the pages
        copy_case("copy_tails", 48, True, 6, 4, 64, 64, "fp16", True),
        # one short sequence branches in two
        branch_case("branch_two", 1, 2, 37, 1, 4, 2, 64, 16, "fp16", False),
        # four beams of each of 32 requests
        branch_case("branch_beams", 32, 4, 1000, 1, 16, 8, 128, 16, "bf16", False),
        # one long prompt sampled 16 times, five drafted tokens in each
        branch_case("branch_samples", 1, 16, 8100, 5, 32, 8, 128, 64, "bf16", False),
        # a few short sequences
        compact_case("compact_small", 4, 200, 4, 2, 64, 16, "fp16", False),
        # a pool of 64 sequences, half of them preempted
        compact_case("compact_pool", 64, 3000, 4, 8, 128, 16, "bf16", False),
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["select", "select", "copy", "branch", "branch", "compact"])
    if op == "select":
        B, W = log(1, 64), log(1, 32)
        V = log(500, 131072)
        while B * W * V > 64 * 4 * 131072:
            B = (B + 1) // 2
        K = rng.choice([W, 2 * W, log(1, 64)])
        return select_case(None, B, W, V, min(K, 64), rng.choice(["bf16", "fp16", "fp32"]),
                           rng.choice([0.0, 0.0, 0.3]), rng.choice([0.0, 0.0, 0.5, 0.9]))
    Hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    page = rng.choice([8, 16, 32, 64, 128])
    layout = dict(Hkv=Hkv, d=d, page=page, dtype=rng.choice(["bf16", "fp16"]), token_rows=rng.random() < 0.3)
    mib = 4.0 * Hkv * page * d / 2 ** 20  # of one page of one layer, K and V
    if op == "copy":
        n = log(1, 500)
        return copy_case(None, n, rng.random() < 0.5, L=max(1, min(log(1, 32), int(500 / (mib * n)))), **layout)
    if op == "branch":
        G = log(1, 32)
        W = log(2, 128 // G)
        return branch_case(None, G, W, log(5, 8000 // G), rng.choice([1, 1, 1, 5, 70]),
                           L=max(1, min(log(1, 16), int(16 / mib))), **layout)
    B, ctx = log(2, 64), log(20, 3000)
    pages = B * (ctx / page + 1)
    return compact_case(None, B, ctx, L=max(1, min(log(1, 16), int(800 / (mib * pages)))), **layout)


# ------------------------------------------------------------------------------------------ inputs
def lengths(c, count):
    """Tokens that each sequence has cached: part of the case's sizes."""
    r = random.Random(count * 7919 + c["ctx"])
    return [r.randint(max(1, c["ctx"] // 2), c["ctx"]) for _ in range(count)]


def pages_of(tokens, page):
    return -(-tokens // page)


def index(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def make_pools(c, pages, generator):
    shape = (c["L"], pages, c["Hkv"], c["page"], c["d"])
    if c["token_rows"]:  # a token's heads side by side within a page
        shape = (c["L"], pages, c["page"], c["Hkv"], c["d"])
    pools = [torch.empty(shape, dtype=TYPES[c["dtype"]], device=DEV).normal_(generator=generator)
             for _ in range(2)]
    return [p.transpose(2, 3) if c["token_rows"] else p for p in pools]


def prepare_select(c, s, g):
    B, W, V = c["B"], c["W"], c["V"]
    x = torch.empty(B, W, V, device=DEV).normal_(generator=g).mul_(3.0)
    if c["masked"]:
        x.masked_fill_(torch.rand(B, W, V, generator=g, device=DEV) < c["masked"], -math.inf)
    s["logits"] = x.to(TYPES[c["dtype"]])
    s["scores"] = -2.0 - 4.0 * torch.rand(B, W, generator=g, device=DEV)
    if c["masked"]:  # some beams found nothing to go on with
        s["scores"].masked_fill_(torch.rand(B, W, generator=g, device=DEV) < 0.1, -math.inf)
    s["finished"] = None
    if c["finished"]:
        s["finished"] = (torch.rand(B, W, generator=g, device=DEV) < c["finished"]).to(torch.uint8)
    s["end"] = V - 1
    return s


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = random.Random(seed)
    s = dict(case=c)
    if c["op"] == "select":
        return prepare_select(c, s, g)
    page = c["page"]
    if c["op"] == "copy":
        ids = list(range(2 * c["n"] + 3))
        host.shuffle(ids)
        s["k"], s["v"] = make_pools(c, len(ids), g)
        s["src"], s["dst"] = index(ids[:c["n"]]), index(ids[c["n"]:2 * c["n"]])
        s["rows"] = index([host.randint(1, page - 1) for _ in range(c["n"])]) if c["tails"] else None
        return s
    if c["op"] == "branch":
        S, live = c["G"] * c["W"], range(0, c["G"] * c["W"], c["W"])
        ctx = dict(zip(live, lengths(c, c["G"])))
        most = max(ctx.values()) + c["n"]
        fresh = S * (pages_of(c["n"], page) + 1)
        s["parents"] = index([b // c["W"] * c["W"] for b in range(S)])
        s["keep"] = index([ctx.get(b, 0) for b in range(S)])
        s["kv_next"] = index([ctx[b // c["W"] * c["W"]] + c["n"] for b in range(S)])
        s["tokens"] = S * c["n"]
        s["places"] = sum(pages_of(ctx[b] + c["n"], page) - ctx[b] // page for b in live) * c["W"]
    else:
        S, live, fresh = c["B"], range(c["B"]), 0
        ctx = dict(zip(live, lengths(c, S)))
        most = max(ctx.values())
        s["turn"] = 0
        s["kv_len"] = index([ctx[b] for b in live])
        for turn in range(2):
            back = [ctx[b] if b % 2 == turn else 0 for b in live]
            s["keep%d" % turn] = index([ctx[b] - back[b] for b in live])
            s["start%d" % turn] = index([0] + list(np.cumsum(back)))
            s["tokens%d" % turn] = sum(back)
            s["places%d" % turn] = sum(pages_of(n, page) for n in back)
    held = {b: pages_of(ctx[b], page) for b in live}
    pool = int(1.1 * (sum(held.values()) + fresh)) + 3
    ids = list(range(pool))
    host.shuffle(ids)
    table = np.full((S, 2 * pages_of(most, page)), -1, dtype=np.int32)
    refs = np.zeros(pool, dtype=np.int32)
    at = 0
    for b in live:
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    refs[ids[:at]] = 1
    s["table"], s["refs"] = torch.from_numpy(table).to(DEV), torch.from_numpy(refs).to(DEV)
    s["k"], s["v"] = make_pools(c, pool, g)
    if c["op"] == "branch":
        s["copies"] = torch.full((3, S), -1, dtype=torch.int32, device=DEV)
    else:
        s["moves"] = torch.full((2, pool // 2), -1, dtype=torch.int32, device=DEV)
        s["count"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------------------------- plain forms
def plain_select(s):
    c = s["case"]
    B, W, V, K = c["B"], c["W"], c["V"], c["K"]
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    total = torch.exp(x - top).double().sum(-1, keepdim=True)
    value = s["scores"].double()[..., None] + (x.double() - (top.double() + torch.log(total)))
    if s["finished"] is not None:
        ended = s["finished"].bool()[..., None]
        end = torch.arange(V, device=DEV) == s["end"]
        value = torch.where(ended, torch.where(end, s["scores"].double()[..., None], -math.inf), value)
    value = torch.where(torch.isfinite(value), value, -math.inf).view(B, W * V)
    if W * V < K:
        value = torch.nn.functional.pad(value, (0, K - W * V), value=-math.inf)
    # the K best: all that are better than the last one and, of its equals, the first
    least = torch.topk(value, K, dim=1).values[:, -1:]
    better, equal = value > least, value == least
    room = K - better.sum(1, keepdim=True)
    taken = better | (equal & (torch.cumsum(equal, 1) <= room))
    at = taken.nonzero()[:, 1].view(B, K)
    best, order = torch.sort(torch.gather(value, 1, at), dim=1, descending=True, stable=True)
    at = torch.gather(at, 1, order)
    there = best > -math.inf
    beam, token = at // V, at % V
    parent = torch.where(there, beam + W * torch.arange(B, device=DEV)[:, None], -1).int()
    token = torch.where(there, token, -1).int()
    done = ~there | (token == s["end"])
    if s["finished"] is not None:
        done = done | torch.gather(s["finished"].bool(), 1, torch.where(there, beam, 0))
    return [best.float(), parent, token, done.to(torch.uint8)]


def plain_copy(k, v, src, dst, rows):
    use = (src >= 0).nonzero().squeeze(1)
    src, dst = src[use].long(), dst[use].long()
    for pool in (k, v):
        new = pool[:, src]
        if rows is not None:
            filled = torch.arange(pool.shape[3], device=DEV) < rows[use][:, None]
            new = torch.where(filled[None, :, None, :, None], new, pool[:, dst])
        pool[:, dst] = new


def plain_free(s, keep):
    table, refs = s["table"], s["refs"]
    place = torch.arange(table.shape[1], device=DEV)
    gone = (place * s["case"]["page"] >= keep[:, None]) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).flatten(), -gone.flatten().int())
    table.masked_fill_(gone, -1)


def plain_fork(s, parents):
    table, refs = s["table"], s["refs"]
    new = torch.where(parents[:, None] >= 0, table[parents.clamp(min=0).long()], -1)
    for t, sign in ((table, -1), (new, 1)):
        refs.index_add_(0, t.clamp(min=0).flatten(), sign * (t >= 0).flatten().int())
    table.copy_(new)


def plain_reserve(s, kv_len, n, places, copies=None):
    """n: new tokens of each sequence; places: how many pages the new tokens' rows lie in."""
    table, refs, page = s["table"], s["refs"], s["case"]["page"]
    kv_len, n = kv_len.long(), n.long()
    ctx = kv_len - n
    first = ctx // page
    count = torch.where(n > 0, (kv_len - 1) // page + 1 - first, 0)
    before = torch.cumsum(count, 0) - count
    seq = torch.repeat_interleave(torch.arange(len(n), device=DEV), count, output_size=places)
    item = torch.arange(places, device=DEV)
    place = item - before[seq] + first[seq]
    entry = table[seq, place].long()
    held, at = entry >= 0, entry.clamp(min=0)
    writers = torch.zeros_like(refs).index_add_(0, at, held.int())
    lowest = torch.full_like(refs, places).long().scatter_reduce_(0, at, torch.where(held, item, places), "amin")
    keep = held & (refs[at] == writers[at]) & (lowest[at] == item)
    need = ~keep
    refs.sub_(writers).index_add_(0, at, keep.int())
    free = (refs == 0).nonzero().squeeze(1)
    page_id = torch.where(need, free[(torch.cumsum(need, 0) - 1).clamp(min=0)], entry)
    table[seq, place] = page_id.int()
    refs.index_add_(0, page_id, need.int())
    if copies is not None:
        at = before.clamp(max=max(places - 1, 0))
        some = (count > 0) & (need & held)[at] & (ctx % page > 0)
        copies[0] = torch.where(some, entry[at], -1).int()
        copies[1] = torch.where(some, page_id[at], -1).int()
        copies[2] = torch.where(some, ctx % page, 0).int()


def plain_branch(s):
    plain_free(s, s["keep"])
    plain_fork(s, s["parents"])
    plain_reserve(s, s["kv_next"], torch.full_like(s["kv_next"], s["case"]["n"]), s["places"], s["copies"])
    plain_copy(s["k"], s["v"], *s["copies"])
    return [s["table"], s["refs"], s["copies"], s["k"], s["v"]]


def plain_compact(s):
    turn = s["turn"]
    s["turn"] = 1 - turn
    plain_free(s, s["keep%d" % turn])
    table, refs = s["table"], s["refs"]
    live = refs != 0
    front = torch.arange(len(refs), device=DEV) < live.sum()
    holes, high = (front & ~live).nonzero().squeeze(1), (~front & live).nonzero().squeeze(1)
    where = torch.arange(len(refs), device=DEV)
    where[high] = holes
    table.copy_(torch.where(table >= 0, where[table.clamp(min=0).long()], -1))
    refs[holes] = refs[high]
    refs[high] = 0
    s["moves"][0, :len(high)] = high.int()
    s["moves"][1, :len(high)] = holes.int()
    s["count"].fill_(len(high))
    plain_copy(s["k"], s["v"], high, holes, None)
    start = s["start%d" % turn]
    plain_reserve(s, s["kv_len"], start[1:] - start[:-1], s["places%d" % turn])
    return [table, refs, s["moves"], s["count"], s["k"], s["v"]]


# ------------------------------------------------------------------------------------- the library
def own_select(s):
    from exact_attention_staged_gb300 import api
    return list(api.beam_select(s["logits"], s["scores"], k=s["case"]["K"], finished=s["finished"],
                                end_token=s["end"]))


def own_branch(s):
    from exact_attention_staged_gb300 import api
    page = s["case"]["page"]
    api.paged_free(s["table"], s["keep"], s["refs"], page)
    api.paged_fork(s["table"], s["parents"], s["refs"])
    api.paged_reserve(s["table"], s["kv_next"], s["refs"], page, tokens=s["tokens"], copies=s["copies"])
    api.paged_copy(s["k"], s["v"], s["copies"][0], s["copies"][1], rows=s["copies"][2])
    return [s["table"], s["refs"], s["copies"], s["k"], s["v"]]


def own_compact(s):
    from exact_attention_staged_gb300 import api
    page, turn = s["case"]["page"], s["turn"]
    s["turn"] = 1 - turn
    api.paged_free(s["table"], s["keep%d" % turn], s["refs"], page)
    api.paged_compact(s["table"], s["refs"], moves=s["moves"], count=s["count"])
    api.paged_copy(s["k"], s["v"], s["moves"][0], s["moves"][1], count=s["count"])
    api.paged_reserve(s["table"], s["kv_len"], s["refs"], page, q_start=s["start%d" % turn],
                      tokens=s["tokens%d" % turn])
    return [s["table"], s["refs"], s["moves"], s["count"], s["k"], s["v"]]


def run(state):
    s = state
    op = s["case"]["op"]
    if op == "copy":
        if own:
            from exact_attention_staged_gb300 import api
            api.paged_copy(s["k"], s["v"], s["src"], s["dst"], rows=s["rows"])
        else:
            plain_copy(s["k"], s["v"], s["src"], s["dst"], s["rows"])
        return [s["k"], s["v"]]
    if own:
        return {"select": own_select, "branch": own_branch, "compact": own_compact}[op](s)
    return {"select": plain_select, "branch": plain_branch, "compact": plain_compact}[op](s)


# -------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "select":
        beams = c["B"] * c["W"]
        read = beams * (1.0 - c["finished"]) * c["V"]  # an ended beam's logits are not needed
        return {"bytes": read * (4 if c["dtype"] == "fp32" else 2) + 5 * beams + 13 * c["B"] * c["K"],
                "flops": 4 * read}
    page = c["page"]
    row = 4 * c["L"] * c["Hkv"] * c["d"]  # K's and V's bytes of one position, all layers
    if c["op"] == "copy":
        r = page / 2 if c["tails"] else page
        return {"bytes": 2 * c["n"] * r * row + (12 if c["tails"] else 8) * c["n"], "flops": 0}
    if c["op"] == "branch":
        G, W, n = c["G"], c["W"], c["n"]
        ctx = lengths(c, G)
        moved = sum(x % page for x in ctx) * (W - 1)  # all but the parent itself copy its last page
        shared = sum(pages_of(x, page) for x in ctx)
        fresh = sum(pages_of(x + n, page) - x // page for x in ctx) * W
        # free: children's entries read and reset; fork: parents' read, children's written; reserve
        entries = 3 * shared * (W - 1) + shared + 2 * fresh
        return {"bytes": 2 * moved * row + 4 * entries + 16 * shared + 8 * fresh + 28 * G * W, "flops": 0}
    ctx = lengths(c, c["B"])
    held = [pages_of(x, page) for x in ctx]
    live, back = sum(held[1::2]), sum(held[::2])
    pool = int(1.1 * (live + back)) + 3
    moved = min(live, back)  # the halves lie one behind the other once both have had a turn
    return {"bytes": 2 * moved * page * row + 4 * (2 * live + 4 * back) + 4 * (pool + 4 * moved) + 8 * back,
            "flops": 0}


# ----------------------------------------------------------------------------------- definitions
def exact_select(c, s):
    B, W, V, K = c["B"], c["W"], c["V"], c["K"]
    scores = torch.full((B, K), -math.inf, dtype=torch.float64, device=DEV)
    parent = torch.full((B, K), -1, dtype=torch.int32, device=DEV)
    token, done = parent.clone(), torch.ones((B, K), dtype=torch.uint8, device=DEV)
    for b in range(B):
        rows = []
        for w in range(W):
            x = s["logits"][b, w].double()
            row = s["scores"][b, w].double() + x - torch.logsumexp(x, 0)
            if s["finished"] is not None and s["finished"][b, w]:
                row = torch.full_like(x, -math.inf)
                row[s["end"]] = s["scores"][b, w].double()
            rows.append(row)
        flat = torch.cat(rows)
        flat[~torch.isfinite(flat)] = -math.inf
        best, at = torch.sort(flat, descending=True, stable=True)
        k = min(K, int((best > -math.inf).sum()))
        scores[b, :k] = best[:k]
        parent[b, :k] = (b * W + at[:k] // V).int()
        token[b, :k] = (at[:k] % V).int()
        ended = token[b, :k] == s["end"]
        if s["finished"] is not None:
            ended |= s["finished"].flatten()[parent[b, :k].long()].bool()
        done[b, :k] = ended.to(torch.uint8)
    return [scores, parent, token, done]


class Pages:
    """Tables and reference counts, one entry at a time."""

    def __init__(self, s):
        self.page = s["case"]["page"]
        self.table = s["table"].cpu().tolist()
        self.refs = s["refs"].cpu().tolist()

    def free(self, keep):
        for row, n in zip(self.table, keep.tolist()):
            for i in range(pages_of(n, self.page), len(row)):
                if row[i] >= 0:
                    self.refs[row[i]] -= 1
                    row[i] = -1

    def fork(self, parents):
        old = [list(row) for row in self.table]
        for b, p in enumerate(parents.tolist()):
            self.table[b] = list(old[p]) if p >= 0 else [-1] * len(old[b])
        self.refs = [0] * len(self.refs)
        for row in self.table:
            for e in row:
                if e >= 0:
                    self.refs[e] += 1

    def reserve(self, kv_len, n):
        copies = [[-1] * len(n), [-1] * len(n), [0] * len(n)]
        writing = [(b, i) for b in range(len(n)) if n[b] > 0
                   for i in range((kv_len[b] - n[b]) // self.page, (kv_len[b] - 1) // self.page + 1)]
        writers = {}
        for b, i in writing:
            writers.setdefault(self.table[b][i], []).append((b, i))
        alone = {w[0] for e, w in writers.items() if e >= 0 and self.refs[e] == len(w)}
        fresh = (e for e in range(len(self.refs)) if self.refs[e] == 0)
        taken = []
        for b, i in writing:
            if (b, i) in alone:
                continue
            old, new = self.table[b][i], next(fresh)
            ctx = kv_len[b] - n[b]
            if old >= 0 and i == ctx // self.page and ctx % self.page:
                copies[0][b], copies[1][b], copies[2][b] = old, new, ctx % self.page
            taken.append((b, i, old, new))
        for b, i, old, new in taken:
            self.table[b][i] = new
            self.refs[new] = 1
            if old >= 0:
                self.refs[old] -= 1
        return copies

    def compact(self):
        live = sum(e != 0 for e in self.refs)
        holes = [e for e in range(live) if self.refs[e] == 0]
        high = [e for e in range(live, len(self.refs)) if self.refs[e] != 0]
        to = dict(zip(high, holes))
        for row in self.table:
            row[:] = [to.get(e, e) for e in row]
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        return high, holes


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "select":
        return exact_select(c, s)
    k, v = s["k"].clone(), s["v"].clone()
    if c["op"] == "copy":
        for i, (a, b) in enumerate(zip(s["src"].tolist(), s["dst"].tolist())):
            r = c["page"] if s["rows"] is None else int(s["rows"][i])
            k[:, b, :, :r], v[:, b, :, :r] = s["k"][:, a, :, :r], s["v"][:, a, :, :r]
        return [k, v]
    pages = Pages(s)
    if c["op"] == "branch":
        pages.free(s["keep"])
        pages.fork(s["parents"])
        kv = s["kv_next"].tolist()
        copies = pages.reserve(kv, [c["n"]] * len(kv))
        for a, b, r in zip(*copies):
            if a >= 0:
                k[:, b, :, :r], v[:, b, :, :r] = s["k"][:, a, :, :r], s["v"][:, a, :, :r]
        return [index(pages.table), index(pages.refs), index(copies), k, v]
    pages.free(s["keep0"])
    high, holes = pages.compact()
    for a, b in zip(high, holes):
        k[:, b], v[:, b] = s["k"][:, a], s["v"][:, a]
    kv = s["kv_len"].tolist()
    pages.reserve(kv, [x if b % 2 == 0 else 0 for b, x in enumerate(kv)])
    moves = s["moves"].clone()
    moves[0, :len(high)], moves[1, :len(high)] = index(high), index(holes)
    return [index(pages.table), index(pages.refs), moves, index([len(high)]), k, v]
