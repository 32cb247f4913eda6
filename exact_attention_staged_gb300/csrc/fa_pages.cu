// fa_pages.cu - the upkeep of paged-cache tables: giving pages to new tokens, forking and freeing
// sequences, moving the live pages together, copying pages.
//
// Sequences may hold the same page; refs counts the table entries (and whatever else the caller
// counts) that hold each page, and a page is free where it is 0.  There is no other state: pages are
// given out lowest id first, so the same calls give the same tables, whatever the order in which
// blocks and atomics run.  Nothing is read back by the host.
//
// The index work is a few bytes per page, bound by the latency of a handful of dependent reads and of the
// launch; copying is bound by HBM.  A step that gives 96 branches back, forks 32 sequences of about 50 pages
// into four each, reserves a page for every new token and copies the 96 shared, part-filled pages in 16
// layers takes 24 us in a row of such steps, of which the copies are about 13: 61 MB, 8.9 us at the copy
// bandwidth, if a source were read once for its three copies; they read it anew each, from L2.
#include "branch.h"
#include "paged.cuh"

#include <algorithm>
#include <climits>
#include <cooperative_groups.h>

namespace fa {
namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ void page_report(int *status, int code = kErrIndex) {
    atomicCAS(status, 0, code);
}

// ------------------------------------------------------------------------------------------ free
// Sequence b keeps the pages of its first keep_len[b] positions.  Every entry behind them is looked
// at (pages may have been reserved ahead): a block takes 1024 of a row, four to a thread.  One round trip to
// the length, one to the table; the counts go down by atomics that nothing waits for.
constexpr int kFreeThreads = 256;
constexpr int kFreeCols = 1024;

__global__ void __launch_bounds__(kFreeThreads) fa_paged_free_kernel(const PagedFreeParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const PageTables &t = p.t;
    const int b = blockIdx.y;
    const long cap = static_cast<long>(t.max_pages) << t.page_shift;
    long keep = p.keep_len[b];
    if (keep < 0 || keep > cap) {
        if (threadIdx.x == 0) page_report(t.status);
        keep = keep < 0 ? 0 : cap;
    }
    const int first = static_cast<int>((keep + (1l << t.page_shift) - 1) >> t.page_shift);
    const long end = min(static_cast<long>(t.max_pages), (blockIdx.x + 1l) * kFreeCols);
    for (long i = blockIdx.x * static_cast<long>(kFreeCols) + threadIdx.x; i < end; i += kFreeThreads) {
        if (i < first) continue;
        int *at = t.table + static_cast<long>(b) * t.max_pages + i;
        const int e = *at;
        if (e == -1) continue;
        *at = -1;
        if (e < 0 || e >= t.num_pages) {
            page_report(t.status);
        } else if (atomicSub(&t.refs[e], 1) <= 0) {  // held by more entries than were counted
            atomicAdd(&t.refs[e], 1);
            page_report(t.status);
        }
    }
}

// ------------------------------------------------------------------------------------------ fork
// Row b becomes row parents[b].  A block takes 2^shift columns of all rows, which are independent of the
// others, into shared memory and writes them back permuted: in place, without a second table.  A page's
// count changes by the row's new holders less one.  Rows that stay as they are and have no other child are
// neither read nor written.  Where an entry is no page, or a count falls below zero, the block looks at its entries
// again once all are counted, reports, and puts to zero what is still below: a count that is too low may be
// below zero on the way, some rows being dropped before others are multiplied.
constexpr int kForkThreads = 256;
constexpr int kForkBatch = 4;  // entries of a thread in flight together

__global__ void __launch_bounds__(kForkThreads) fa_paged_fork_kernel(const PagedForkParams p) {
    extern __shared__ int fork_smem[];
    const PageTables &t = p.t;
    const int B = t.B, shift = p.shift;
    int *parent = fork_smem, *children = fork_smem + B, *tile = fork_smem + 2 * B;
    for (int b = threadIdx.x; b < B; b += kForkThreads) children[b] = 0;
    griddep_launch_dependents();
    griddep_wait();
    __syncthreads();
    for (int b = threadIdx.x; b < B; b += kForkThreads) {
        int q = p.parents[b];
        if (q < -1 || q >= B) {
            if (blockIdx.x == 0) page_report(t.status);
            q = b;
        }
        parent[b] = q;
        if (q >= 0) atomicAdd(&children[q], 1);
    }
    __syncthreads();
    if (blockIdx.x == 0 && p.kv_len != nullptr) {
        int *len = tile;  // before the columns use it
        for (int b = threadIdx.x; b < B; b += kForkThreads) len[b] = p.kv_len[b];
        __syncthreads();
        for (int b = threadIdx.x; b < B; b += kForkThreads)
            if (parent[b] != b) p.kv_len[b] = parent[b] >= 0 ? len[parent[b]] : 0;
        __syncthreads();
    }
    const int c0 = blockIdx.x << shift, c = threadIdx.x & ((1 << shift) - 1);
    const int width = min(1 << shift, t.max_pages - c0), entries = B << shift;
    // entry x is column c of row x >> shift, and so are the thread's others
    auto used = [&](int x) {
        const int b = x >> shift;
        return x < entries && c < width && !(parent[b] == b && children[b] == 1);
    };
    auto place = [&](int x) { return static_cast<long>(x >> shift) * t.max_pages + c0 + c; };
    auto real = [&](int e) { return e >= 0 && e < t.num_pages; };
    bool bad = false;
    for (int x0 = threadIdx.x; x0 < entries; x0 += kForkBatch * kForkThreads) {
        int e[kForkBatch];
#pragma unroll
        for (int k = 0; k < kForkBatch; ++k) {
            const int x = x0 + k * kForkThreads;
            if (used(x)) e[k] = t.table[place(x)];
        }
#pragma unroll
        for (int k = 0; k < kForkBatch; ++k) {
            const int x = x0 + k * kForkThreads;
            if (!used(x)) continue;
            tile[x] = e[k];
            const int more = children[x >> shift] - 1;
            bad |= static_cast<unsigned>(e[k]) + 1 > static_cast<unsigned>(t.num_pages);  // -1: none
            if (more != 0 && real(e[k])) bad |= atomicAdd(&t.refs[e[k]], more) + more < 0;
        }
    }
    if (__builtin_expect(__syncthreads_or(bad), 0)) {  // out of the way: in the loop below it took 2 us of 12 more
#pragma unroll 1
        for (int x = threadIdx.x; x < entries; x += kForkThreads) {
            if (!used(x) || tile[x] == -1) continue;
            if (!real(tile[x]) || (children[x >> shift] != 1 && atomicMax(&t.refs[tile[x]], 0) < 0))
                page_report(t.status);
        }
    }
    for (int x = threadIdx.x; x < entries; x += kForkThreads) {
        if (!used(x)) continue;
        const int b = x >> shift, q = parent[b];
        if (q == b) continue;
        const int now = q >= 0 ? tile[(q << shift) + c] : -1;
        if (now != tile[x]) t.table[place(x)] = now;
    }
}

// --------------------------------------------------------------------------------------- reserve
// One cluster does all of it (a CTA where there is little), in steps with a barrier between them.
// An item is a page place that a sequence's new tokens write to; items are numbered by sequence,
// then place, and so are the pages that they get.
//   1  items are numbered, free pages are listed by rank, as many as there are items
//   2  every item that has a page gives its hold back: refs becomes the holders that do not write
//   3  where none is left, the items that had the page compete for it with their numbers
//   4  the lowest keeps it; all other items, and those that had none, are numbered again
//   5  and take the page of their rank
// A step is a round trip to L2 and a barrier, some 0.7 us; a thread keeps one item in registers.  All of refs is read,
// whatever the number of items: a page for each of 128 sequences takes 6.5 us of a pool of 8000 pages, 10.8 of
// 100000 and 17.6 of 260000.
constexpr int kReserveThreads = 1024;
constexpr int kReserveCtas = 8;    // the portable cluster size
constexpr int kReserveRounds = 8;  // groups of four pages whose state a thread keeps

// Exclusive prefix of x over the CTA's threads, and the sum; `scratch` holds 33 ints.
__device__ __forceinline__ int block_scan(int x, int *scratch, int *sum) {
    const int lane = lane_id(), w = warp_id();
    int upto = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    __syncthreads();  // the scratch of the call before has been read
    if (lane == 31) scratch[w] = upto;
    __syncthreads();
    if (w == 0) {
        const int n = static_cast<int>(blockDim.x >> 5);
        int v = lane < n ? scratch[lane] : 0, s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane < n) scratch[lane] = s - v;
        if (lane == 31) scratch[32] = s;
    }
    __syncthreads();
    *sum = scratch[32];
    return scratch[w] + upto - x;
}

// Whether refs of the four pages from i on (0 behind the end) make them free, as bits.
__device__ __forceinline__ int free_bits(const int *refs, long i, long end) {
    if (i >= end) return 0;
    int r[4] = {1, 1, 1, 1};
    if (i + 4 <= end) {
        const int4 v = __ldcg(reinterpret_cast<const int4 *>(refs + i));
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else {
        for (int k = 0; i + k < end; ++k) r[k] = __ldcg(refs + i + k);
    }
    return (r[0] == 0) | (r[1] == 0) << 1 | (r[2] == 0) << 2 | (r[3] == 0) << 3;
}

// A sequence's first place, and how many its tokens write to.
__device__ __forceinline__ int reserve_places(const PagedReserveParams &p, int b, bool report, int *first,
                                              int *ctx) {
    const PagedSeq s = paged_seq(p.c, b);
    *ctx = max(s.ctx, 0);
    *first = *ctx >> p.t.page_shift;
    if (s.bad && report) page_report(p.t.status);
    if (s.bad || s.n == 0 || s.len == 0) return 0;
    return ((s.len - 1) >> p.t.page_shift) + 1 - *first;
}

// Offsets in order are what bounds the items by the batch's tokens: with others nothing is reserved.
__device__ __forceinline__ bool reserve_ordered(const PagedReserveParams &p, bool first_cta) {
    bool ordered = true;
    for (int b = threadIdx.x; b < p.t.B; b += blockDim.x) {
        if (p.c.q_start != nullptr && p.c.q_start[b + 1] < p.c.q_start[b]) ordered = false;
        if (p.copies != nullptr && first_cta) {
            p.copies[b] = p.copies[p.t.B + b] = -1;
            p.copies[2 * p.t.B + b] = 0;
        }
    }
    if (__syncthreads_and(ordered) != 0) return true;
    if (threadIdx.x == 0 && first_cta) page_report(p.t.status);
    return false;
}

// No more items than threads, and no more pages than their registers hold.
__global__ void __launch_bounds__(kReserveThreads) fa_paged_reserve_kernel(const PagedReserveParams p) {
    extern __shared__ int before[];  // [B + 1] items before each sequence's
    __shared__ int scratch[33];
    __shared__ int counts[2];               // this CTA's free pages and needs
    __shared__ int low;                     // 1: some page has more entries than were counted
    __shared__ int fresh[kReserveThreads];  // free pages of ranks cta * threads on
    griddep_launch_dependents();
    griddep_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const PageTables &t = p.t;
    const int B = t.B, tid = threadIdx.x, threads = static_cast<int>(blockDim.x);
    const int cta = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
    auto barrier = [&] {
        if (ctas > 1) cluster.sync();
        else __syncthreads();
    };
    // a thread keeps the state of `rounds` neighbouring groups of four pages
    const int rounds = static_cast<int>(((t.num_pages + 3l) / 4 + threads * ctas - 1) / (threads * ctas));
    const long from = 4l * rounds * (cta * threads + tid);
    unsigned free_of = 0;
#pragma unroll
    for (int r = 0; r < kReserveRounds; ++r)
        if (r < rounds)
            free_of |= static_cast<unsigned>(free_bits(t.refs, from + 4 * r, t.num_pages)) << 4 * r;
    if (!reserve_ordered(p, cta == 0)) return;
    // items and free pages before this thread's: with the first sequences in one scan, frees in the lower half
    int items = 0, frees = 0, free_mine = 0, sum;
    for (int b0 = 0; b0 < B; b0 += threads) {
        const int b = b0 + tid;
        int first, ctx;
        const unsigned n = b < B ? reserve_places(p, b, cta == 0, &first, &ctx) : 0;
        const unsigned x = block_scan(n << 16 | (b0 == 0 ? __popc(free_of) : 0), scratch, &sum);
        if (b < B) before[b] = items + static_cast<int>(x >> 16);
        items += static_cast<int>(static_cast<unsigned>(sum) >> 16);
        if (b0 == 0) frees = sum & 0xffff, free_mine = static_cast<int>(x & 0xffff);
    }
    if (tid == 0) {
        before[B] = items;
        counts[0] = frees;
        low = 0;
    }
    barrier();
    int free_before = free_mine, free_all = 0;
    for (int c = 0; c < ctas; ++c) {
        const int x = *cluster.map_shared_rank(&counts[0], c);
        if (c < cta) free_before += x;
        free_all += x;
    }
    for (unsigned bits = free_of; bits != 0 && free_before < items; bits &= bits - 1, ++free_before)
        *cluster.map_shared_rank(&fresh[free_before % threads], free_before / threads) =
            static_cast<int>(from) + __ffs(static_cast<int>(bits)) - 1;

    const int g = cta * threads + tid;  // this thread's item
    int b = 0, e = -1, held = 1, *at = nullptr;
    bool had = false, bad = false;
    if (g < items) {
        int r = B;  // before[b] <= g < before[r]
        while (r - b > 1) {
            const int m = (b + r) / 2;
            if (before[m] <= g) b = m;
            else r = m;
        }
        const int place = (max(paged_seq(p.c, b).ctx, 0) >> t.page_shift) + g - before[b];
        at = t.table + static_cast<long>(b) * t.max_pages + min(place, t.max_pages - 1);
        e = *at;
        had = e >= 0 && e < t.num_pages;
        if (had) held = atomicSub(&t.refs[e], 1);
        else bad = e != -1;
    }
    barrier();
    if (had && __ldcg(&t.refs[e]) <= 0) atomicMin(&t.refs[e], INT_MIN + g);
    barrier();
    bool need = g < items;
    if (had && __ldcg(&t.refs[e]) == INT_MIN + g) {
        t.refs[e] = 1;
        need = false;
    }
    // items before this one that need a page, and, in the upper half, those whose page was held by more entries
    // than were counted (the barriers do not wait for `held` so)
    int rank = block_scan(need | (held <= 0) << 16, scratch, &sum);
    rank &= 0xffff;
    bad |= held <= 0;
    if (tid == 0) counts[1] = sum & 0xffff;
    if (sum >> 16 != 0)
#pragma unroll 1
        for (int c = 0; c < ctas; ++c) *cluster.map_shared_rank(&low, c) = 1;
    barrier();
    int page = -1;
    auto fresh_page = [&](int r) { return *cluster.map_shared_rank(&fresh[r % threads], r / threads); };
    if (need) {
        for (int c = 0; c < cta; ++c) rank += *cluster.map_shared_rank(&counts[1], c);
        if (low == 0 && rank < free_all) page = fresh_page(rank);
    }
    if (__builtin_expect(low != 0, 0)) {
        // A page that was listed as free may be kept by an item by now, and is left out.  There are enough others,
        // as that item needs none.
#pragma unroll 1
        for (int r = 0, left = rank; need && r < min(items, free_all); ++r) {
            const int id = fresh_page(r);
            if (__ldcg(&t.refs[id]) == 0 && left-- == 0) {
                page = id;
                break;
            }
        }
        barrier();  // nobody takes a page while others look
    }
    if (need) {
        *at = page;
        if (page >= 0) {
            t.refs[page] = 1;
            const int rows = max(paged_seq(p.c, b).ctx, 0) & ((1 << t.page_shift) - 1);
            if (had && p.copies != nullptr && g == before[b] && rows > 0) {
                p.copies[b] = e;
                p.copies[B + b] = page;
                p.copies[2 * B + b] = rows;
            }
        } else {
            page_report(t.status, kErrFull);
        }
    }
    if (bad) page_report(t.status);
    if (ctas > 1) cluster.sync();  // the others have read this CTA's shared memory
}

// Any number of items and pages: the same steps, in which every thread walks its share and finds it anew, and
// free pages are counted and listed (in the workspace) once it is known how many are needed.  A page for each of 128
// sequences from a pool of 300000 takes 19 us, of 1000000 32; 5000 pages 22 and 16384 54; prompts of 8000 tokens in
// pages of 16, 64 of them (32000 pages) 30, 256 of them 96.
__global__ void __launch_bounds__(kReserveThreads) fa_paged_reserve_many_kernel(const PagedReserveParams p) {
    extern __shared__ int before[];  // [B + 1] items before each sequence's
    __shared__ int scratch[33];
    __shared__ int counts[2];        // this CTA's needs and free pages
    griddep_launch_dependents();
    griddep_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const PageTables &t = p.t;
    const int B = t.B, tid = threadIdx.x;
    const int cta = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());

    if (!reserve_ordered(p, cta == 0)) return;
    int items = 0;
    for (int b0 = 0; b0 < B; b0 += kReserveThreads) {
        const int b = b0 + tid;
        int first, ctx, sum;
        const int x = block_scan(b < B ? reserve_places(p, b, cta == 0, &first, &ctx) : 0, scratch, &sum);
        if (b < B) before[b] = items + x;
        items += sum;
    }
    if (tid == 0) before[B] = items;
    __syncthreads();
    const int per = (items + ctas - 1) / ctas;
    const int lo = min(items, cta * per), hi = min(items, lo + per);
    // the sequence of item g, and its entry
    auto find = [&](int g, int *b) {
        int l = 0, r = B;  // before[l] <= g < before[r]
        while (r - l > 1) {
            const int m = (l + r) / 2;
            if (before[m] <= g) l = m;
            else r = m;
        }
        *b = l;
        const PagedSeq s = paged_seq(p.c, l);
        const int place = (max(s.ctx, 0) >> t.page_shift) + g - before[l];
        return t.table + static_cast<long>(l) * t.max_pages + min(place, t.max_pages - 1);
    };

    for (int g = lo + tid; g < hi; g += kReserveThreads) {
        int b;
        const int e = *find(g, &b);
        if (e >= 0 && e < t.num_pages) {
            if (atomicSub(&t.refs[e], 1) <= 0) page_report(t.status);  // more entries than were counted
        } else if (e != -1) {
            page_report(t.status);
        }
    }
    cluster.sync();
    for (int g = lo + tid; g < hi; g += kReserveThreads) {
        int b;
        const int e = *find(g, &b);
        if (e >= 0 && e < t.num_pages && __ldcg(&t.refs[e]) <= 0) atomicMin(&t.refs[e], INT_MIN + g);
    }
    cluster.sync();
    int needs = 0;
    for (int g = lo + tid; g < hi; g += kReserveThreads) {
        int b;
        int *at = find(g, &b);
        const int e = *at;
        const bool had = e >= 0 && e < t.num_pages;
        if (had && __ldcg(&t.refs[e]) == INT_MIN + g) {
            t.refs[e] = 1;
            continue;
        }
        ++needs;
        *at = -1;
        if (had && p.copies != nullptr && g == before[b]) {
            const int rows = max(paged_seq(p.c, b).ctx, 0) & ((1 << t.page_shift) - 1);
            if (rows > 0) {
                p.copies[b] = e;
                p.copies[2 * B + b] = rows;
            }
        }
    }
    // this CTA's share of the pool, in whole groups of four pages
    const long share = ((t.num_pages + 3l) / 4 + ctas - 1) / ctas * 4;
    const long from = min(static_cast<long>(t.num_pages), cta * share);
    const long to = min(static_cast<long>(t.num_pages), from + share);
    int frees = 0;
    for (long i = from + 4 * tid; i < to; i += 4 * kReserveThreads) frees += __popc(free_bits(t.refs, i, to));
    int sum;
    block_scan(needs, scratch, &sum);
    if (tid == 0) counts[0] = sum;
    block_scan(frees, scratch, &sum);
    if (tid == 0) counts[1] = sum;
    cluster.sync();
    int need_before = 0, need_all = 0, free_before = 0, free_all = 0;
    for (int c = 0; c < ctas; ++c) {
        const int *other = cluster.map_shared_rank(counts, c);
        if (c < cta) need_before += other[0], free_before += other[1];
        need_all += other[0], free_all += other[1];
    }
    for (long i0 = from; i0 < to && free_before < need_all; i0 += 4 * kReserveThreads) {
        const long i = i0 + 4 * tid;
        const int bits = free_bits(t.refs, i, to);
        int rank = free_before + block_scan(__popc(bits), scratch, &sum);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (bits >> k & 1) {
                if (rank < need_all) p.fresh[rank] = static_cast<int>(i + k);
                ++rank;
            }
        free_before += sum;
    }
    cluster.sync();  // also: nobody's counts are read any more
    for (int g0 = lo; g0 < hi; g0 += kReserveThreads) {
        const int g = g0 + tid;
        int b = 0, *at = nullptr;
        if (g < hi) at = find(g, &b);
        const bool need = at != nullptr && *at == -1;
        const int rank = need_before + block_scan(need, scratch, &sum);
        need_before += sum;
        if (!need) continue;
        const int page = rank < free_all ? __ldcg(&p.fresh[rank]) : -1;
        const bool copied = p.copies != nullptr && g == before[b] && __ldcg(&p.copies[b]) >= 0;
        if (page >= 0) {
            *at = page;
            t.refs[page] = 1;
            if (copied) p.copies[B + b] = page;
        } else {
            page_report(t.status, kErrFull);
            if (copied) {
                p.copies[b] = -1;
                p.copies[2 * B + b] = 0;
            }
        }
    }
}

// --------------------------------------------------------------------------------------- compact
// n live pages; the k-th live page at or behind n moves to the k-th free page before n.  With
// live(i) the live pages before i, a free page i < n is number i - live(i) of the free ones, and a
// live page i >= n makes move live(i) - live(n).  Both lists ascend, so a table's entry finds its move by
// bisection.
__device__ __forceinline__ void compact_apply(const PagedCompactParams &p, int moves, long me, long threads) {
    const PageTables &t = p.t;
    for (long i = me; i < moves; i += threads) {
        const int from = __ldcg(&p.src[i]);
        t.refs[__ldcg(&p.dst[i])] = t.refs[from];
        t.refs[from] = 0;
    }
    const int first = moves > 0 ? __ldcg(&p.src[0]) : t.num_pages;
    const long entries = static_cast<long>(t.B) * t.max_pages;
    for (long i = me; i < entries; i += threads) {
        const int e = t.table[i];
        if (e < first && e >= -1) continue;
        int lo = 0, hi = moves;  // src[lo] <= e < src[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (__ldcg(&p.src[mid]) <= e) lo = mid;
            else hi = mid;
        }
        if (e >= first && moves > 0 && __ldcg(&p.src[lo]) == e) t.table[i] = __ldcg(&p.dst[lo]);
        else page_report(t.status);  // no page, or one that nobody holds
    }
}

// The lists, and, where p.apply is set (a single CTA), what follows from them.
__global__ void __launch_bounds__(kReserveThreads) fa_paged_compact_kernel(const PagedCompactParams p) {
    __shared__ int scratch[33];
    __shared__ int counts[2];  // this CTA's live pages; those of them before n
    griddep_launch_dependents();
    griddep_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const PageTables &t = p.t;
    const int tid = threadIdx.x;
    const int cta = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
    const long share = ((t.num_pages + 3l) / 4 + ctas - 1) / ctas * 4;
    const long from = min(static_cast<long>(t.num_pages), cta * share);
    const long to = min(static_cast<long>(t.num_pages), from + share);
    auto live_of = [&](long i, long end) {
        const int there = static_cast<int>(max(0l, min(4l, end - i)));
        return there - __popc(free_bits(t.refs, i, end));
    };
    int sum, mine = 0;
    for (long i = from + 4 * tid; i < to; i += 4 * kReserveThreads) mine += live_of(i, to);
    block_scan(mine, scratch, &sum);
    if (tid == 0) counts[0] = sum;
    cluster.sync();
    int n = 0, live = 0;  // live pages in all, and before this CTA's share
    for (int c = 0; c < ctas; ++c) {
        const int x = cluster.map_shared_rank(counts, c)[0];
        n += x;
        if (c < cta) live += x;
    }
    mine = 0;
    const long border = min(to, static_cast<long>(n));
    for (long i = from + 4 * tid; i < border; i += 4 * kReserveThreads) mine += live_of(i, border);
    block_scan(mine, scratch, &sum);
    if (tid == 0) counts[1] = sum;
    cluster.sync();
    int front = 0;  // live pages before n
    for (int c = 0; c < ctas; ++c) front += cluster.map_shared_rank(counts, c)[1];
    if (cta == 0 && tid == 0) *p.count = n - front;
    for (long i0 = from; i0 < to; i0 += 4 * kReserveThreads) {
        const long i = i0 + 4 * tid;
        const int bits = free_bits(t.refs, i, to);
        int at = live + block_scan(live_of(i, to), scratch, &sum);
        for (int k = 0; k < 4 && i + k < to; ++k) {
            const int id = static_cast<int>(i + k);
            const bool is_free = bits >> k & 1;
            if (id < n && is_free) p.dst[id - at] = id;
            if (id >= n && !is_free) p.src[at - front] = id;
            if (!is_free) ++at;
        }
        live += sum;
    }
    cluster.sync();  // the lists are there, and nobody's counts are read any more
    if (p.apply) compact_apply(p, n - front, tid, kReserveThreads);
}

__global__ void __launch_bounds__(256) fa_paged_apply_kernel(const PagedCompactParams p) {
    griddep_launch_dependents();
    griddep_wait();
    compact_apply(p, *p.count, blockIdx.x * 256l + threadIdx.x, gridDim.x * 256l);
}

// ------------------------------------------------------------------------------------------ copy
// A run is consecutive 16-byte pieces of one page of one layer: a head's rows or, where the heads of a token lie
// side by side, a row's heads.  A block takes some of the runs of one pair of pages, so that the pair is
// looked up once, and a warp as many runs at a time as give each lane four pieces in flight (48 copies of up to 63 rows
// of 4 x 64 in 6 layers take 5.0 us; 7.4 with eight pieces, 9.7 with a run per warp).
constexpr int kCopyWarps = 8;
constexpr int kCopyBatch = 4;  // pieces of a lane in flight together

__global__ void __launch_bounds__(kCopyWarps * 32) fa_paged_copy_kernel(const PagedCopyParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int n = p.count != nullptr ? min(max(*p.count, 0), p.n) : p.n;
    const unsigned parts = p.parts, per = p.per;  // blocks of a pair, and the runs that each takes
    const long units = static_cast<long>(n) * parts;
    for (long u = blockIdx.x; u < units; u += gridDim.x) {
        const int e = static_cast<int>(u / parts);
        const unsigned part = static_cast<unsigned>(u - static_cast<long>(e) * parts);
        const int src = p.src[e], dst = p.dst[e];
        const int rows = p.rows != nullptr ? p.rows[e] : p.page_size;
        if (src < 0 || dst < 0) continue;
        if (src >= p.num_pages || dst >= p.num_pages || rows < 0 || rows > p.page_size) {
            if (threadIdx.x == 0) page_report(p.status);
            continue;
        }
        // runs of a layer's K or V, in order (layer, K or V, run)
        const unsigned runs = p.rows_inner ? p.heads : rows;
        const int pieces = (p.rows_inner ? rows : p.heads) << p.piece_shift;
        const unsigned end = min((part + 1) * per, static_cast<unsigned>(p.L) * 2 * runs);
        int lanes = 32;  // of a run
        while (lanes > 1 && lanes / 2 * kCopyBatch >= pieces) lanes /= 2;
        const int at_once = 32 / lanes, part_lane = lane_id() & (lanes - 1);
        for (unsigned x = part * per + warp_id() * at_once + lane_id() / lanes; x < end; x += kCopyWarps * at_once) {
            const unsigned slab = x / runs, run = x - slab * runs;
            const PagedCopySide &s = slab & 1 ? p.v : p.k;
            const uint16_t *from = s.base + (slab >> 1) * s.layer + src * s.page + run * s.outer;
            const long over = (dst - static_cast<long>(src)) * s.page;
            auto place = [&](int i) {
                return const_cast<uint16_t *>(from) + (i >> p.piece_shift) * s.inner +
                       (i & ((1 << p.piece_shift) - 1)) * 8;
            };
            for (int i0 = part_lane; i0 < pieces; i0 += lanes * kCopyBatch) {
                uint4 v[kCopyBatch];
#pragma unroll
                for (int k = 0; k < kCopyBatch; ++k) {
                    const int i = i0 + lanes * k;
                    if (i < pieces) v[k] = *reinterpret_cast<const uint4 *>(place(i));
                }
#pragma unroll
                for (int k = 0; k < kCopyBatch; ++k) {
                    const int i = i0 + lanes * k;
                    if (i < pieces) *reinterpret_cast<uint4 *>(place(i) + over) = v[k];
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_paged_free(const PagedFreeParams &p, cudaStream_t stream) {
    const dim3 grid((p.t.max_pages - 1) / kFreeCols + 1, p.t.B);
    return launch_overlapped(fa_paged_free_kernel, grid, kFreeThreads, 0, stream, p);
}

cudaError_t launch_paged_fork(PagedForkParams p, cudaStream_t stream) {
    // columns of a block: a thousand entries or so, a sector of every row at least where that fits
    p.shift = 5;
    while (p.shift > 0 && (static_cast<long>(p.t.B) << p.shift) > (p.shift > 3 ? 1024 : 24 * 1024)) --p.shift;
    const size_t bytes = sizeof(int) * p.t.B * (2 + (1ul << p.shift));
    if (bytes > 48 * 1024) {
        // most with one column of all sequences, or with the last that have two
        constexpr int kMost = static_cast<int>(sizeof(int)) * 3 * kBranchMaxSeqs;
        static_assert(kMost >= static_cast<int>(sizeof(int)) * (2 * 24 * 1024 / 2 + 24 * 1024));
        static std::atomic<unsigned long long> ready{0};
        const cudaError_t e =
            allow_smem(ready, reinterpret_cast<const void *>(fa_paged_fork_kernel), kMost, p.t.device);
        if (e != cudaSuccess) return e;
    }
    return launch_overlapped(fa_paged_fork_kernel, dim3(((p.t.max_pages - 1) >> p.shift) + 1), kForkThreads,
                             bytes, stream, p);
}

// Threads of each CTA and CTAs that hold the items and pages in registers, or {0, 0}.
ReserveShape reserve_shape(int T, int B, int num_pages, int page_size) {
    const long items = static_cast<long>(T) / page_size + 2l * B;
    for (const ReserveShape s : {ReserveShape{256, 1}, ReserveShape{1024, 1}, ReserveShape{1024, kReserveCtas}}) {
        const long all = static_cast<long>(s.threads) * s.ctas;
        if (items <= all && num_pages <= 4 * kReserveRounds * all) return s;
    }
    return {0, 0};
}

cudaError_t launch_paged_reserve(const PagedReserveParams &p, cudaStream_t stream) {
    const size_t smem = sizeof(int) * (p.t.B + 1);
    const ReserveShape s = reserve_shape(p.c.T, p.t.B, p.t.num_pages, 1 << p.t.page_shift);
    // up to 4096 sequences (two items each): 16 KB, beside 5
    if (s.threads > 0) return launch_clusters(fa_paged_reserve_kernel, 1, s.ctas, s.threads, smem, stream, p);
    if (smem > 32 * 1024) {
        static std::atomic<unsigned long long> ready{0};
        const cudaError_t e = allow_smem(ready, reinterpret_cast<const void *>(fa_paged_reserve_many_kernel),
                                         sizeof(int) * (kBranchMaxSeqs + 1), p.t.device);
        if (e != cudaSuccess) return e;
    }
    return launch_clusters(fa_paged_reserve_many_kernel, 1, kReserveCtas, kReserveThreads, smem, stream, p);
}

cudaError_t launch_paged_compact(PagedCompactParams p, cudaStream_t stream) {
    // Small pools and tables take one CTA, which applies the lists too: eight pages and entries of a thread at
    // most (24000 entries of a pool of 17000 pages take 7 us more in the same launch).
    const long entries = static_cast<long>(p.t.B) * p.t.max_pages, most = std::max(entries, p.t.num_pages + 0l);
    p.apply = most <= 8 * kReserveThreads ? 1 : 0;
    const cudaError_t e = launch_clusters(fa_paged_compact_kernel, 1, p.apply ? 1 : kReserveCtas, kReserveThreads,
                                          0, stream, p);
    if (e != cudaSuccess || p.apply) return e;
    const long blocks = std::min((most + 255) / 256, 152l * 8);
    return launch_overlapped(fa_paged_apply_kernel, dim3(static_cast<unsigned>(blocks)), 256, 0, stream, p);
}

cudaError_t launch_paged_copy(PagedCopyParams p, cudaStream_t stream) {
    // blocks of 32 KB or so (a full page's), of less where the pairs are few
    const long runs = 2l * p.L * (p.rows_inner ? p.heads : p.page_size);
    const long pieces = static_cast<long>(p.rows_inner ? p.page_size : p.heads) << p.piece_shift;
    long per = std::max(2048l / pieces, static_cast<long>(kCopyWarps));
    while (per > kCopyWarps && p.n * ((runs + per - 1) / per) < 152 * 8) per /= 2;
    p.per = static_cast<unsigned>(per);
    p.parts = static_cast<unsigned>((runs + per - 1) / per);
    // Many short-lived blocks balance best (half of a pool moved in 358 us with 128 per SM, 360 with 64, 368
    // with 32), but with a count on the device most may find nothing to do.
    const long blocks = std::min(static_cast<long>(p.n) * p.parts, 152l * (p.count != nullptr ? 64 : 128));
    return launch_overlapped(fa_paged_copy_kernel, dim3(static_cast<unsigned>(blocks)), kCopyWarps * 32, 0,
                             stream, p);
}

}  // namespace fa
