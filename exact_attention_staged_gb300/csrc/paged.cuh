// paged.cuh - how the paged-cache kernels find a sequence's tokens and pages.  Host code uses the
// same functions to check tables before a call, so what the device refuses and what the host
// reports are one rule.
#pragma once

#include "fa_internal.h"

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

#ifdef __CUDACC__
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
