// paged.cuh - how the paged-cache kernels find a sequence's tokens and pages.  Host code uses the
// same functions to check tables before a call, so what the device refuses and what the host
// reports are one rule.
#pragma once

#include "positions.h"

namespace fa {

// One sequence's share of the batch.  `bad`: a stored value was out of range (and was clamped).
struct PagedSeq {
    int tok0;  // its first token in the batch
    int n;     // its new tokens
    int len;   // its cached positions, the new tokens included
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
// unit_cost + tile_cost * tiles of it (tiles at least 1), where tile_cost is 2 for a unit of two
// query tiles and 1 for a unit of one.  CTA c of G takes [c W / G, (c + 1) W / G) of the line's
// length W, so every CTA gets an equal share whatever the mixture of lengths.  A border inside a
// unit cuts it between two key tiles; its pieces are merged afterwards.
constexpr int kPagedKeys = 128;  // keys per tile

struct PagedWork {
    int tile_toks;  // tokens of one query tile
    int unit_toks;  // tokens per unit: one or two query tiles
    int unit_cost;
    int causal;
};

// sum of floor((a i + b) / m) for i < n (a, b >= 0): Euclid's steps on the lattice points below
// the line, a handful of divisions.
__host__ __device__ inline long paged_floor_sum(long n, long m, long a, long b) {
    long sum = 0;
    while (n > 0) {
        if (a >= m) {
            sum += n * (n - 1) / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            sum += n * (b / m);
            b %= m;
        }
        const long y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const long t = m;
        m = a;
        a = t;
    }
    return sum;
}

__host__ __device__ inline int paged_units(const PagedSeq &s, const PagedWork &w) {
    return (s.n + w.unit_toks - 1) / w.unit_toks;  // per K/V head
}
__host__ __device__ inline int paged_tile_cost(const PagedWork &w, int toks) {
    return toks > w.tile_toks ? 2 : 1;
}
// Key tiles that the first `toks` new tokens of a sequence see.
__host__ __device__ inline int paged_tiles(const PagedSeq &s, const PagedWork &w, int toks) {
    const int end = w.causal ? s.len - s.n + toks : s.len;
    return end > 0 ? (end + kPagedKeys - 1) / kPagedKeys : 0;
}

// Length on the line of the first i units of one K/V head.
__host__ __device__ inline long paged_prefix(const PagedSeq &s, const PagedWork &w, long i) {
    const long last = paged_units(s, w) - 1;
    const long m = i < last ? i : last;  // units before the last one: whole ones
    long tiles = 0;
    if (m > 0) {
        if (w.causal) {  // unit j sees len - n + (j + 1) unit_toks keys, at least a weight of 1
            const long ctx = static_cast<long>(s.len) - s.n;
            long none = ctx < 0 ? -ctx / w.unit_toks : 0;
            if (none > m) none = m;
            tiles = none + paged_floor_sum(m - none, kPagedKeys, w.unit_toks,
                                           ctx + (none + 1) * w.unit_toks + kPagedKeys - 1);
        } else {
            const int t = paged_tiles(s, w, 0);
            tiles = m * (t > 0 ? t : 1);
        }
    }
    long sum = m * w.unit_cost + tiles * paged_tile_cost(w, w.unit_toks);
    if (i > last) {
        const int t = paged_tiles(s, w, s.n);
        sum += w.unit_cost + (t > 0 ? t : 1) * paged_tile_cost(w, s.n - static_cast<int>(last) * w.unit_toks);
    }
    return sum;
}

// What a unit costs beside its tiles (Q, the first loads, the epilogue), in single tiles; units of
// up to two query tiles or of one.
__host__ __device__ inline int paged_unit_cost(int tiles) { return tiles == 2 ? 2 : 0; }

// CTAs that share a line of length W: no stretch shorter than two single key tiles, which is one
// step of a CTA's two softmax groups (and no shorter than a tile of two query tiles, so that every
// CTA between a unit's first and last one has a piece of it).
__host__ __device__ inline int paged_ctas(long total, int most) {
    const long g = total / 2;
    return g >= most ? most : g > 0 ? static_cast<int>(g) : total > 0 ? 1 : 0;
}
__host__ __device__ inline long paged_border(long total, int ctas, int c) {
    return total * c / ctas;
}

// A stretch of one unit's key tiles, [t0, t1) of `tiles` (tiles at least 1).
struct PagedPiece {
    int tok0;     // first token, in the batch
    int toks;     // tokens of the unit
    int kvh;
    int b;
    int last0;    // last key that the first token sees (that token j sees: + j when causal)
    int len;
    int t0, t1, tiles;
    long unit_end;  // end of the unit on the line, from the position before it was taken
};

struct PagedCursor {
    PagedSeq s;
    int b, g, i;  // sequence, K/V head and unit
    int at;       // place inside the unit's length

    // `pos`: length inside sequence b that lies before the position
    __host__ __device__ void start(const PagedView &c, const PagedWork &w, int seq, long pos) {
        b = seq;
        s = paged_seq(c, b);
        const int units = paged_units(s, w);
        const long each = paged_prefix(s, w, units);
        g = static_cast<int>(pos / each);
        pos -= g * each;
        int lo = 0, hi = units - 1;  // the last unit whose prefix is <= pos
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (paged_prefix(s, w, mid) <= pos)
                lo = mid;
            else
                hi = mid - 1;
        }
        i = lo;
        at = static_cast<int>(lo > 0 ? pos - paged_prefix(s, w, lo) : pos);
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
        p.last0 = w.causal ? s.len - s.n + i0 : s.len - 1;
        p.len = s.len;
        const int seen = paged_tiles(s, w, i0 + p.toks), cost = paged_tile_cost(w, p.toks);
        p.tiles = seen > 0 ? seen : 1;
        const int length = w.unit_cost + cost * p.tiles;
        p.unit_end = length - at;
        auto tile_of = [&](int x) { return x > w.unit_cost ? (x - w.unit_cost) / cost : 0; };
        p.t0 = tile_of(at);
        if (room < length - at) {
            at += static_cast<int>(room);
            room = 0;
            p.t1 = tile_of(at);
            return p;
        }
        p.t1 = p.tiles;
        room -= length - at;
        at = 0;
        if (++i == paged_units(s, w)) {
            i = 0;
            if (++g == c.Hkv) {
                g = 0;
                do {
                    if (++b >= c.B) break;
                    s = paged_seq(c, b);
                } while (s.n == 0);
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

__device__ __forceinline__ void paged_report(const PagedView &c) {
    atomicExch(c.status, kErrIndex);
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
