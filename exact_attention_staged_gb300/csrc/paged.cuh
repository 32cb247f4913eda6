// paged.cuh - how the paged-cache kernels find a sequence's tokens and pages.  Host code uses the
// same functions to check tables before a call, so what the device refuses and what the host
// reports are one rule.
#pragma once

#include "positions.h"

namespace fa {

// One sequence's share of the batch.  `bad`: a stored value was out of range (and was clamped).
struct PagedSeq {
    int tok0;  // its first token in the batch
    int n;     // its new tokens, no more than max_q
    int len;   // its cached positions, the new tokens included
    int ctx;   // place of its first new token (below 0: before the sequence), whatever max_q cuts off
    bool bad;
};

__host__ __device__ inline PagedSeq paged_seq_of(int first, int next, int len, int T, int max_q,
                                                 long cap) {
    PagedSeq s;
    s.bad = false;
    auto clamp = [&](long x, long lo, long hi) {
        if (x < lo) { s.bad = true; return lo; }
        if (x > hi) { s.bad = true; return hi; }
        return x;
    };
    s.tok0 = static_cast<int>(clamp(first, 0, T));
    const long end = clamp(next, s.tok0, T);
    s.n = static_cast<int>(clamp(end - s.tok0, 0, max_q));
    s.len = static_cast<int>(clamp(len, 0, cap));
    s.ctx = s.len - static_cast<int>(end - s.tok0);
    return s;
}

__host__ __device__ inline PagedSeq paged_seq(const PagedView &c, int b) {
    const long cap = static_cast<long>(c.max_pages) << c.page_shift;
    const int each = c.T / c.B;
    const int first = c.q_start != nullptr ? c.q_start[b] : b * each;
    const int next = c.q_start != nullptr ? c.q_start[b + 1] : first + each;
    return paged_seq_of(first, next, c.kv_len[b], c.T, c.max_q, cap);
}

// The page that holds position pos (inside the sequence's length), or -1 when the table's entry
// is no page of this cache.
__host__ __device__ inline int paged_page(const PagedView &c, int b, int pos) {
    const int i = pos >> c.page_shift;
    if (pos < 0 || i >= c.max_pages) return -1;
    const int id = c.table[static_cast<long>(b) * c.max_pages + i];
    return id >= 0 && id < c.num_pages ? id : -1;
}

// ------------------------------------------------------------------------------------------
// How the attention's work is cut.  A unit is one K/V head of one sequence with up to
// `unit_toks` of its new tokens (all query heads of the group), walked over the key tiles that its
// last token sees.  Units in order (sequence, K/V head, tokens) form one line; a unit takes
// unit_cost + tile_cost * keys of it (keys at least 1), where tile_cost is 2 for a unit of two
// query tiles and 1 for a unit of one.  The line is cut into one equal stretch per CTA, whatever
// the mixture of lengths.  A border inside a unit cuts it between two key tiles; its pieces are
// merged afterwards.  Lengths go by keys and not by tiles because their sums over units are then
// polynomials: a CTA finds its place with a few multiplications (with rounded tiles the search
// took up to 13000 cycles before the first load).
constexpr int kPagedKeys = 128;  // keys per tile

struct PagedWork {
    int tile_toks;  // tokens of one query tile
    int unit_toks;  // tokens per unit: one or two query tiles
    int unit_cost;
    int causal;
};

// What a unit costs beside its keys (Q, the first loads, the epilogue): for units of up to two query
// tiles as much as 2.5 of their key tiles (a whole 8k prompt, whose first units are short, takes
// 414 us with one tile, 391 with 1.75, 371 with 2.5, 368 with 3.5 and 372 with 5; two chunks of
// 1k at d = 64 28.4, 28.0, 29.2, 29.5 and 30.3); units of one tile load ahead into the next.
__host__ __device__ inline int paged_unit_cost(int tiles) { return tiles == 2 ? 640 : 0; }

__host__ __device__ inline int paged_units(const PagedSeq &s, const PagedWork &w) {
    return s.n <= w.unit_toks ? (s.n > 0 ? 1 : 0) : (s.n - 1) / w.unit_toks + 1;  // per K/V head
}
__host__ __device__ inline int paged_tile_cost(const PagedWork &w, int toks) {
    return toks > w.tile_toks ? 2 : 1;
}
// Keys that the first `toks` new tokens of a sequence see.
__host__ __device__ inline int paged_keys(const PagedSeq &s, const PagedWork &w, int toks) {
    const int end = w.causal ? s.ctx + toks : s.len;
    return end > 0 ? end : 0;
}

// Length on the line of the first m units of one K/V head, all but the last of which are whole.
__host__ __device__ inline long paged_prefix(const PagedSeq &s, const PagedWork &w, long m) {
    long keys;
    if (w.causal) {  // unit j sees ctx + (j + 1) unit_toks keys, at least a weight of 1
        const long ctx = s.ctx;
        long none = 0;
        if (ctx < 0) {
            none = -ctx / w.unit_toks;
            if (none > m) none = m;
        }
        keys = none + (m - none) * ctx +
               w.unit_toks * (m * (m + 1) / 2 - none * (none + 1) / 2);
    } else {
        keys = m * (s.len > 0 ? s.len : 1);
    }
    return m * w.unit_cost + keys * paged_tile_cost(w, w.unit_toks);
}
// Keys of a unit as the line counts them: at least one; a sequence's only unit (generated or drafted
// tokens) by whole tiles, so that borders fall on tiles where there are few of them.
__host__ __device__ inline long paged_line_keys(int keys, int units) {
    if (units > 1) return keys > 0 ? keys : 1;
    return keys > 0 ? (static_cast<long>(keys) + kPagedKeys - 1) / kPagedKeys * kPagedKeys : kPagedKeys;
}
__host__ __device__ inline long paged_head(const PagedSeq &s, const PagedWork &w) {
    const int units = paged_units(s, w);
    if (units == 0) return 0;
    return (units > 1 ? paged_prefix(s, w, units - 1) : 0) + w.unit_cost +
           paged_line_keys(paged_keys(s, w, s.n), units) *
               paged_tile_cost(w, s.n - (units - 1) * w.unit_toks);
}

// The line of length `total` cut for up to `most` CTAs: the first r of them take q + 1, the others q.
// No stretch is shorter than a unit's cost and two single key tiles, one step of a CTA's two softmax
// groups (so none is without work, and every CTA between a cut unit's first and last one has a
// piece of it).
// Where every sequence is one unit per K/V head and there are no more units than CTAs, cutting them is
// left out when it would not pay: a CTA takes a whole unit, nothing is merged.  By unit, the time is
// that of the longest unit (1950 cycles a key tile) or of HBM for all of them (2570 cycles a tile
// and 152 SMs); as a line it is HBM's plus about 9000 cycles for cutting and merging.  16 x 8 heads of
// 8k keys: 83.4 us by unit, 88.4 as a line; of 4k to 8k keys: 74.3 and 69.8.  The cycles are those of
// d = 128; a tile of d = 64 has half the bytes, and there the rule takes whole units too often: 14 x 8
// heads of 8k keys 49.3 us by unit, 45.0 as a line, 16 x 8 50.7 and 50.2, 18 x 8 52.8 and 57.0.
struct PagedLine {
    long total, q;
    int ctas, r;
    bool by_unit;
    // longest: length of the longest head; heads: K/V heads of sequences with new tokens
    __host__ __device__ void cut(long length, long longest, long heads, const PagedWork &w, int most) {
        const int least = w.unit_cost + 2 * kPagedKeys;
        total = length;
        by_unit = w.unit_toks == w.tile_toks && heads <= most && 115 * longest <= length + 68000;
        if (by_unit) {
            total = heads;
            ctas = static_cast<int>(heads);
            q = heads > 0 ? 1 : 0;
            r = 0;
            return;
        }
        ctas = length >= static_cast<long>(most) * least ? most
               : length >= least ? static_cast<int>(length) / least : length > 0 ? 1 : 0;
        if (ctas == 0) {
            q = r = 0;
        } else if (length < (1l << 31)) {
            q = static_cast<unsigned>(length) / static_cast<unsigned>(ctas);
            r = static_cast<int>(length - q * ctas);
        } else {
            q = length / ctas;
            r = static_cast<int>(length - q * ctas);
        }
    }
    __host__ __device__ long border(int c) const { return q * c + (c < r ? c : r); }
    // The CTA whose stretch holds position x.
    __host__ __device__ int holder(long x) const {
        const long wide = (q + 1) * r;
        return static_cast<int>(x < wide ? x / (q + 1) : r + (x - wide) / q);
    }
};

// A stretch of one unit's key tiles, [t0, t1) of `tiles` (tiles at least 1).
struct PagedPiece {
    int tok0;     // first token, in the batch
    int toks;     // tokens of the unit
    int kvh;
    int b;
    int last0;    // last key that the first token sees (that token j sees: + j when causal)
    int len;
    int t0, t1, tiles;
    long left;    // of the unit on the line, from where the piece was taken
};

struct PagedCursor {
    PagedSeq s;
    int b, g, i, units;  // sequence, K/V head, unit; units per head
    long at;             // place inside the unit's length

    // `pos`: length inside sequence seq that lies before the position; `each`: its length per
    // K/V head.  Head and unit are estimated in floating point and put right by the exact lengths.
    __host__ __device__ void start(const PagedView &c, const PagedWork &w, int seq,
                                   const PagedSeq &which, long each, long pos) {
        b = seq;
        s = which;
        units = paged_units(s, w);
        g = static_cast<int>(static_cast<float>(pos) / static_cast<float>(each));
        if (g > c.Hkv - 1) g = c.Hkv - 1;
        while (g * each > pos) --g;
        while (g + 1 < c.Hkv && (g + 1) * each <= pos) ++g;
        pos -= g * each;
        i = 0;
        if (units > 1) {  // the last unit whose prefix is <= pos; pos = a i^2 + f i while ctx >= 0
            const long ctx = s.ctx;
            const float cost = static_cast<float>(paged_tile_cost(w, w.unit_toks));
            const float a = w.causal ? 0.5f * cost * w.unit_toks : 0.f;
            const float f = w.unit_cost + cost * (w.causal ? ctx + 0.5f * w.unit_toks
                                                           : static_cast<float>(s.len));
            const float x = static_cast<float>(pos);
            int lo = 0, hi = units - 1, tries = 0;
            int mid = ctx >= 0 ? static_cast<int>(2.f * x / (f + sqrtf(f * f + 4.f * a * x))) : hi / 2;
            long before = 0;
            while (lo < hi) {
                mid = mid <= lo ? lo + 1 : mid > hi ? hi : mid;
                const long here = paged_prefix(s, w, mid);
                if (here <= pos) {
                    lo = mid;
                    before = here;
                    ++mid;
                } else {
                    hi = mid - 1;
                    mid = hi;
                }
                if (++tries > 4) mid = lo + (hi - lo + 1) / 2;  // the estimate was no help
            }
            i = lo;
            pos -= before;
        }
        at = pos;
    }
    // The next piece, taking at most `room` of the line; `room` is lowered by what it took.  The
    // piece is empty (t0 == t1) where both borders fall before or into the same key tile.
    __host__ __device__ PagedPiece take(const PagedView &c, const PagedWork &w, long &room) {
        PagedPiece p;
        const int i0 = i * w.unit_toks;
        p.tok0 = s.tok0 + i0;
        p.toks = s.n - i0 < w.unit_toks ? s.n - i0 : w.unit_toks;
        p.kvh = g;
        p.b = b;
        p.last0 = w.causal ? s.ctx + i0 : s.len - 1;
        p.len = s.len;
        const int cost = paged_tile_cost(w, p.toks);
        const long keys = paged_line_keys(paged_keys(s, w, i0 + p.toks), units);
        p.tiles = static_cast<int>((keys - 1) / kPagedKeys) + 1;
        const long length = w.unit_cost + cost * keys;
        p.left = length - at;
        auto tile_of = [&](long x) {
            return x > w.unit_cost ? static_cast<int>((x - w.unit_cost) >> (cost == 2 ? 8 : 7)) : 0;
        };
        p.t0 = tile_of(at);
        if (room < p.left) {
            at += room;
            room = 0;
            p.t1 = tile_of(at);
            return p;
        }
        p.t1 = p.tiles;
        room -= p.left;
        at = 0;
        if (++i == units) {
            i = 0;
            if (++g == c.Hkv) {
                g = 0;
                do {
                    if (++b >= c.B) break;
                    s = paged_seq(c, b);
                } while (s.n == 0);
                units = paged_units(s, w);
            }
        }
        return p;
    }
};

#ifdef __CUDACC__
// TMA: 4-D tiled load of one box into shared memory, completing on an mbarrier with its bytes.
__device__ __forceinline__ void tma_load_4d(void *smem_dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// A wait that ran out leaves outputs undefined and a bad index does not: it keeps the status word.
__device__ __forceinline__ void paged_report(const PagedView &c) {
    atomicCAS(c.status, 0, kErrIndex);
}

// Sequence of token t: the b with q_start[b] <= t < q_start[b + 1], or -1 (a token before the
// first or behind the last sequence).  The whole warp calls it; each step narrows the range to
// one of 32 parts, so a batch of up to 1024 sequences takes two reads.
__device__ __forceinline__ int paged_find(const PagedView &c, int t) {
    if (c.q_start == nullptr) return t / (c.T / c.B);
    const int lane = static_cast<int>(threadIdx.x & 31);
    int lo = 0, hi = c.B;  // b + 1 lies in (lo, hi], or nothing does
    if (c.q_start[0] > t) return -1;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int i = min(lo + (lane + 1) * step, hi);
        const unsigned past = __ballot_sync(0xffffffffu, c.q_start[i] <= t);
        if (past == 0xffffffffu) return -1;  // every sequence ends at or before t
        const int k = __popc(past);
        hi = min(lo + (k + 1) * step, hi);
        lo = min(lo + k * step, hi - 1);  // below hi even when the offsets are not in order
        if (step == 1) return lo;
    }
    return -1;
}
#endif

}  // namespace fa
