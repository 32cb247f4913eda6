// fa_paged_attn.cu - attention of the new tokens of every sequence over its paged cache, sm_103a.
//
// Row i of the n new tokens of sequence b sees the keys j <= kv_len[b] - n + i (causal) or all
// kv_len[b] of them: O = softmax(scale q K^T) V and the logsumexp, by the online softmax
// (FlashAttention-2 reading notes, Algorithm 1) with the statistic merge of the FlashAttention
// paper detail, Technique 1, for units whose keys are spread over several CTAs.
//
// Rows.  The query heads of a K/V head's group share its keys, so a query tile of 128 rows is
// floor(128 / rep) tokens times the rep heads of one group: one TMA box of the token-major Q.  A
// prompt chunk's unit is two such tiles (256 rows per K/V tile read from L2, as in the forward); a
// batch whose sequences bring no more than one tile of tokens runs the one-tile form, which has
// room for more K/V tiles in flight and is bound by reading the cache.
//
// Keys.  A tile is 128 positions, whatever the page size: its pages are loaded by one TMA box each
// into their rows of the 128-byte-swizzled tile (a page of 8 rows or more starts on a swizzle
// atom); pages behind the sequence's end are loaded from an index outside the pool, which TMA
// fills with zeros.  Scores behind the end are masked, and V's rows between the end and the end of
// its page are zeroed in shared memory before the product, so that whatever the cache holds there
// (NaN included) meets a probability of zero as a zero.
//
// Work.  paged.cuh cuts the line of all units' key tiles into one equal stretch per CTA, on the
// device (the host knows no lengths), so prompt chunks and single tokens of any mixture balance,
// and a single sequence's keys spread over all SMs.  A tile costs about the same either way: two
// query tiles' products and softmax take about 2900 cycles per 64 KB of K and V, and 64 KB is
// what HBM brings one SM in about 2700.
//
// Warps: 0 loads and walks the units, 1 issues the MMAs, four per query tile run the softmax.  With
// two query tiles the MMA order per key tile is PV_0(j-1), S_0(j), PV_1(j-1), S_1(j) as in the
// forward; with one, S has two buffers and S(j+1) is issued before PV(j) as in decode.
#include "paged.cuh"

#include <type_traits>

namespace fa {
namespace {

template <int D, int TILES>
struct PagedLayout {
    static constexpr int kTileBytes = 128 * D * 2;  // one 128 x d tile of 16-bit values
    static constexpr int kBoxes = D / 64;
    static constexpr int kBoxBytes = 128 * 128;
    static constexpr int kSlots = D == 128 ? (TILES == 2 ? 5 : 6) : 12;  // K/V ring
    static constexpr int kSlotOff = TILES * kTileBytes;                  // after the Q tiles
    static constexpr int kBarOff = kSlotOff + kSlots * kTileBytes;
    // q_full, q_empty, full[S], empty[S], s_full[2], p_full[2], o_final[2], pv_done,
    // unit_full[2], unit_empty[2], drain
    static constexpr int kNumBars = 2 + 2 * kSlots + 12;
    static constexpr int kUnitOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;  // two unit slots
    static constexpr int kScanOff = kUnitOff + 2 * 32;  // the plan's sums: 16 longs
    static constexpr int kMiscOff = kScanOff + 16 * 8;  // TMEM base, abort flag
    static constexpr int kBytes = kMiscOff + 8;
    static constexpr int kAlloc = kBytes + 1024;
    static constexpr int kThreads = TILES == 2 ? 384 : 192;
    static constexpr int kSoftWarp = TILES == 2 ? 4 : 2;  // first softmax warp
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kAlloc <= 232448, "shared memory per CTA");
};

template <bool BF16>
using elem_t = typename std::conditional<BF16, __nv_bfloat16, __half>::type;

// Natural logsumexp of a row from its max (log2 units) and sum; a sum that is NaN stays one.
__device__ __forceinline__ float row_lse(float m, float l) {
    if (l == 0.f) return -INFINITY;
    return l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : l;
}

// A unit's piece as the load warp hands it to the others (one of two slots in shared memory).
struct PieceSlot {
    int tok0;   // first token, in the batch; -1: no more pieces
    int toks;
    int kvh;
    int last0;  // last key that the first token sees
    int len;
    int t0, t1; // key tiles, t1 not beyond what the unit sees
    int dest;   // -1: O and LSE, otherwise the slot of its partial result
};

// Key tiles of the piece that query tile q takes part in: [t0, first tile it does not see).
__device__ __forceinline__ int piece_end(const PieceSlot &u, int q, int tile_toks, int causal) {
    const int toks = min(u.toks - q * tile_toks, tile_toks);
    if (toks <= 0) return u.t0;
    const int last = u.last0 + (causal ? q * tile_toks + toks - 1 : 0);
    const int end = last >= 0 ? last / kPagedKeys + 1 : 0;
    return max(u.t0, min(u.t1, end));
}

// The CTA's stretch of the line of key tiles, found by all threads together: W is the sum of the
// sequences' weights; the border W c / G is then looked for in a running sum over the sequences.
struct Stretch {
    long total;     // W
    int ctas;       // G: CTAs that get work
    long begin, end;
    int seq;        // sequence that holds `begin`, and the weight before it
    long before;
};
template <int THREADS>
__device__ __forceinline__ Stretch find_stretch(const PagedAttnParams &p, const PagedWork &w,
                                                long *scan) {
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    constexpr int kWarps = THREADS / 32;
    auto weight = [&](int b) -> long {
        if (b >= p.c.B) return 0;
        const PagedSeq s = paged_seq(p.c, b);
        if (s.bad && blockIdx.x == 0) paged_report(p.c);
        return s.n > 0 ? p.c.Hkv * paged_prefix(s, w, paged_units(s, w)) : 0;
    };
    long mine = 0, first = weight(tid);  // the first THREADS sequences' weights are kept
    for (int b = tid; b < p.c.B; b += THREADS) mine += b == tid ? first : weight(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) scan[warp] = mine;
    __syncthreads();
    Stretch r;
    r.total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) r.total += scan[i];
    r.ctas = static_cast<int>(min(static_cast<long>(gridDim.x), r.total));
    const int c = static_cast<int>(blockIdx.x);
    r.begin = r.end = 0;
    r.seq = 0;
    r.before = 0;
    if (c >= r.ctas) return r;
    r.begin = paged_border(r.total, r.ctas, c);
    r.end = paged_border(r.total, r.ctas, c + 1);
    long base = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += THREADS) {  // inclusive sums of THREADS sequences at a time
        const long x = b0 == 0 ? first : weight(b0 + tid);
        long sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        __syncthreads();  // the sums read above are done with
        if (lane == 31) scan[warp] = sum;
        __syncthreads();
        long all = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) sum += scan[i];
            all += scan[i];
        }
        if (base + all > r.begin) {
            __syncthreads();
            if (base + sum - x <= r.begin && r.begin < base + sum) {
                scan[0] = b0 + tid;
                scan[1] = base + sum - x;
            }
            __syncthreads();
            r.seq = static_cast<int>(scan[0]);
            r.before = scan[1];
            break;
        }
        base += all;
    }
    return r;
}

template <int D, bool BF16, int TILES>
__global__ void __launch_bounds__(PagedLayout<D, TILES>::kThreads, 1)
    fa_paged_attn_kernel(const __grid_constant__ PagedMaps maps, const PagedAttnParams p) {
    using L = PagedLayout<D, TILES>;
    constexpr uint32_t kIdescS = idesc_f16(128, 128, BF16, false);
    constexpr uint32_t kIdescPV = idesc_f16(128, D, BF16, true);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *q_full = bars, *q_empty = bars + 1;
    uint64_t *full = bars + 2, *empty = full + L::kSlots;
    uint64_t *s_full = empty + L::kSlots;  // [2]: per query tile, or per S buffer
    uint64_t *p_full = s_full + 2;         // [2]: the same
    uint64_t *o_final = p_full + 2;        // [2]: per query tile
    uint64_t *pv_done = o_final + 2;
    uint64_t *unit_full = pv_done + 1, *unit_empty = unit_full + 2;  // [2] each
    uint64_t *drain = unit_empty + 2;
    volatile int *unit_slot = reinterpret_cast<volatile int *>(smem + L::kUnitOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMiscOff + 4);
    const int warp = warp_id(), lane = lane_id();
    const PagedWork work = {TILES * p.tile_toks, p.causal};

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < L::kSlots; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);  // one arrival per softmax warp of a query tile
            mbar_init(&o_final[i], 1);
            mbar_init(&unit_full[i], 1);
            mbar_init(&unit_empty[i], 1 + 4 * TILES);  // the MMA warp and the softmax warps
        }
        mbar_init(pv_done, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, L::kTmemCols);
        tmem_relinquish();
    }
    const Stretch mine =
        find_stretch<L::kThreads>(p, work, reinterpret_cast<long *>(smem + L::kScanOff));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // the merge queued after this grid may take its place early; it waits for this grid's end
    if (threadIdx.x == 0) griddep_launch_dependents();

    auto read_slot = [&](int e) {
        PieceSlot u;
        volatile int *s = unit_slot + 8 * e;
        u.tok0 = s[0];
        u.toks = s[1];
        u.kvh = s[2];
        u.last0 = s[3];
        u.len = s[4];
        u.t0 = s[5];
        u.t1 = s[6];
        u.dest = s[7];
        return u;
    };

    if (warp < L::kSoftWarp) {
        if constexpr (TILES == 2) regs_dec<80>();
        if (warp == 0) {
            // ---------------------------------------------------------------- load warp
            const int shift = p.c.page_shift;
            const int box_rows = min(1 << shift, kPagedKeys);  // rows of one page in a tile
            const int boxes = kPagedKeys / box_rows;           // pages of a tile
            int n = 0;   // K/V tiles issued into the ring
            int nq = 0;  // Q loads issued
            bool ok = true;
            PagedCursor cur;
            long at = mine.begin;
            if (at < mine.end) cur.start(p.c, work, mine.seq, at - mine.before);
            int4 cut0 = make_int4(-1, 0, 0, 0);  // what the merge has to do for this CTA
            int cut_n = 0;
            for (int k = 0;; ++k) {
                const int e = k & 1;
                if (k >= 2 && !mbar_wait_warp(&unit_empty[e], ((k >> 1) - 1) & 1, p.ctl,
                                              abort_flag)) {
                    ok = false;
                    break;
                }
                if (at >= mine.end) {
                    if (lane == 0) {
                        unit_slot[8 * e] = -1;
                        mbar_arrive(&unit_full[e]);
                    }
                    break;
                }
                const PagedPiece u = cur.take(p.c, work, mine.end - at);
                const bool whole = u.t1 - u.t0 == u.weight;
                if (!whole && u.t0 == 0) {  // starts a unit that other CTAs finish
                    const long unit_end = at + u.weight;
                    const int c1 = static_cast<int>(
                        (unit_end * mine.ctas + mine.total - 1) / mine.total - 1);
                    cut0 = make_int4(u.tok0, u.toks, u.kvh, 0);
                    cut_n = c1 - static_cast<int>(blockIdx.x) + 1;
                }
                at += u.t1 - u.t0;
                // what the unit really sees: nothing, if it stands before its sequence
                const int seen = u.last0 + (p.causal ? u.toks - 1 : 0) < 0 ? u.t0 : u.t1;
                if (lane == 0) {
                    volatile int *s = unit_slot + 8 * e;
                    s[0] = u.tok0;
                    s[1] = u.toks;
                    s[2] = u.kvh;
                    s[3] = u.last0;
                    s[4] = u.len;
                    s[5] = u.t0;
                    s[6] = seen;
                    s[7] = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (u.t0 == 0 ? 1 : 0);
                    __threadfence_block();
                    mbar_arrive(&unit_full[e]);
                }
                auto load_q = [&]() {  // the Q tiles are free once the last unit's last S is done
                    if (nq > 0 && !mbar_wait_warp(q_empty, (nq - 1) & 1, p.ctl, abort_flag))
                        return false;
                    if (lane == 0) {
                        const int tiles = TILES == 2 && u.toks > p.tile_toks ? 2 : 1;
                        mbar_arrive_expect_tx(
                            q_full, tiles * L::kBoxes * 128 * p.rep * p.q_box_toks);
                        for (int t = 0; t < tiles; ++t)
                            for (int b = 0; b < L::kBoxes; ++b)
                                tma_load_4d(smem + t * L::kTileBytes + b * L::kBoxBytes, &maps.q,
                                            b * 64, 0, u.kvh, u.tok0 + t * p.tile_toks, q_full);
                    }
                    ++nq;
                    return true;
                };
                // page ids of the piece, 32 at a time in the lanes, the next 32 read ahead
                const int *row = p.c.table + static_cast<long>(u.b) * p.c.max_pages;
                const int have = (u.len + (1 << shift) - 1) >> shift;  // pages of the sequence
                auto ids = [&](int first) {
                    const int i = first + lane;
                    return i < have ? row[i] : p.c.num_pages;  // outside the pool: zeros
                };
                int base = ((u.t0 * kPagedKeys) >> shift) & ~31;
                int now = ids(base), next = ids(base + 32);
                bool q_done = false;
                for (int j = u.t0; j < seen && ok; ++j) {
                    const int page0 = (j * kPagedKeys) >> shift;
                    if (page0 >= base + 32) {
                        base += 32;
                        now = next;
                        next = ids(base + 32);
                    }
                    int id = __shfl_sync(0xffffffffu, now, (page0 - base + lane) & 31);
                    if (lane < boxes && (id < 0 || id > p.c.num_pages ||
                                         (id == p.c.num_pages && page0 + lane < have))) {
                        paged_report(p.c);
                        id = p.c.num_pages;
                    }
                    const int y = (j * kPagedKeys) & ((1 << shift) - 1);
                    for (int kv = 0; kv < 2; ++kv) {
                        const int s = n % L::kSlots;
                        if (!mbar_wait_warp(&empty[s], ((n / L::kSlots) & 1) ^ 1, p.ctl,
                                            abort_flag)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(&full[s], L::kTileBytes);
                        __syncwarp();
                        if (lane < boxes) {
                            uint8_t *dst = smem + L::kSlotOff + s * L::kTileBytes +
                                           lane * box_rows * 128;
                            for (int b = 0; b < L::kBoxes; ++b)
                                tma_load_4d(dst + b * L::kBoxBytes, kv ? &maps.v : &maps.k, b * 64,
                                            maps.rows_inner ? y : u.kvh,
                                            maps.rows_inner ? u.kvh : y, id, &full[s]);
                        }
                        ++n;
                    }
                    // the first K/V pair goes ahead of Q: its slots free before the Q tiles do
                    if (ok && !q_done) {
                        ok = load_q();
                        q_done = true;
                    }
                }
                if (ok && !q_done) ok = load_q();  // a unit that sees nothing takes its turn
                if (!ok) break;
            }
            if (p.cut != nullptr && lane == 0) {
                p.cut[2 * blockIdx.x] = cut0;
                p.cut[2 * blockIdx.x + 1] = make_int4(cut_n, 0, 0, 0);
            }
            if (!ok || *abort_flag) {
                // let every copy still in flight land before shared memory goes away
                if (lane == 0) {
                    if (nq > 0) drain_wait(q_full, (nq - 1) & 1, p.ctl);
                    for (int l = n > L::kSlots ? n - L::kSlots : 0; l < n; ++l)
                        drain_wait(&full[l % L::kSlots], (l / L::kSlots) & 1, p.ctl);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ---------------------------------------------------------------- MMA issuer
            const SDesc dq0 = sdesc_make(smem_u32(smem), 16, 1024);                 // Q: K-major
            const SDesc dk0 = sdesc_make(smem_u32(smem + L::kSlotOff), 16, 1024);   // K: K-major
            const SDesc dv0 = sdesc_make(smem_u32(smem + L::kSlotOff), L::kBoxBytes,
                                         1024);                                      // V: MN-major
            auto issue_s = [&](int q, int buf, int ks) {
                const SDesc a = sdesc_add(dq0, q * L::kTileBytes);
                const SDesc b = sdesc_add(dk0, ks * L::kTileBytes);
                if constexpr (D == 128)
                    mma_ss_chain_k128(tmem + buf * 128, a, b, kIdescS, 0u);
                else
                    mma_ss_chain_k64(tmem + buf * 128, a, b, kIdescS, 0u);
            };
            auto issue_pv = [&](int q, int buf, int vs, bool accumulate) {
                mma_ts_chain_k128(tmem + 256 + q * D, tmem + buf * 128,
                                  sdesc_add(dv0, vs * L::kTileBytes), kIdescPV,
                                  accumulate ? 1u : 0u);
            };
            // V of key tile j in slot vs has landed; its rows from the sequence's end to the end
            // of that page become zeros (pages behind it were loaded as zeros)
            auto clear_tail = [&](int len, int j, int vs) {
                const int r0 = len - j * kPagedKeys;
                if (r0 >= kPagedKeys) return;
                const int size = 1 << p.c.page_shift;
                const int r1 = min(kPagedKeys, (r0 + size - 1) & ~(size - 1));
                uint8_t *tile = smem + L::kSlotOff + vs * L::kTileBytes;
                for (int b = 0; b < L::kBoxes; ++b)
                    for (int x = r0 * 128 + lane * 16; x < r1 * 128; x += 512)
                        *reinterpret_cast<uint4 *>(tile + b * L::kBoxBytes + x) =
                            make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
            };
            int n = 0;              // K/V tiles consumed from the ring
            int pcnt[2] = {0, 0};   // PV products per query tile (TILES == 2)
            int g = 0;              // key tiles consumed (TILES == 1): S buffer g % 2
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int e = k & 1;
                if (!mbar_wait_warp(&unit_full[e], (k >> 1) & 1, p.ctl, abort_flag)) {
                    ok = false;
                    break;
                }
                const PieceSlot u = read_slot(e);
                if (u.tok0 < 0) break;
                if (!mbar_wait_warp(q_full, k & 1, p.ctl, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if constexpr (TILES == 2) {
                    const int end0 = piece_end(u, 0, p.tile_toks, p.causal);
                    const int end1 = piece_end(u, 1, p.tile_toks, p.causal);
                    const int last = max(end0, end1) - 1;
                    const int p0[2] = {pcnt[0], pcnt[1]};
                    for (int j = u.t0; ok && j <= last + 1; ++j) {
                        const int ks = n % L::kSlots;  // of tile j; V of tile j - 1 is one before
                        const int vs = (n + L::kSlots - 1) % L::kSlots;
                        if (j <= last) {
                            if (!mbar_wait_warp(&full[ks], (n / L::kSlots) & 1, p.ctl,
                                                abort_flag)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                        }
                        bool v_ready = false;
                        for (int t = 0; t < 2 && ok; ++t) {
                            const int end = t ? end1 : end0;
                            if (j > u.t0 && j - 1 < end) {
                                if (!v_ready) {
                                    if (!mbar_wait_warp(&full[vs], ((n - 1) / L::kSlots) & 1,
                                                        p.ctl, abort_flag)) {
                                        ok = false;
                                        break;
                                    }
                                    clear_tail(u.len, j - 1, vs);
                                    v_ready = true;
                                }
                                if (!mbar_wait_warp(&p_full[t], pcnt[t] & 1, p.ctl, abort_flag)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                issue_pv(t, t, vs, pcnt[t] > p0[t]);
                                ++pcnt[t];
                            }
                            if (j < end) {
                                issue_s(t, t, ks);
                                umma_commit_el(&s_full[t]);
                            }
                        }
                        if (!ok) break;
                        if (j == last) umma_commit_el(q_empty);
                        if (j > u.t0) umma_commit_el(&empty[vs]);
                        if (j <= last) {
                            umma_commit_el(&empty[ks]);
                            n += 2;
                        }
                    }
                    if (!ok) break;
                    if (last < u.t0) umma_commit_el(q_empty);  // nothing seen: Q is free at once
                    for (int t = 0; t < 2; ++t)
                        if (pcnt[t] > p0[t]) umma_commit_el(&o_final[t]);
                } else {
                    const int end = piece_end(u, 0, p.tile_toks, p.causal);
                    auto next_s = [&](int j) -> bool {
                        const int x = n + 2 * (j - u.t0), ks = x % L::kSlots, gg = g + j - u.t0;
                        if (!mbar_wait_warp(&full[ks], (x / L::kSlots) & 1, p.ctl, abort_flag))
                            return false;
                        tc_fence_after();
                        issue_s(0, gg & 1, ks);
                        umma_commit_el(&s_full[gg & 1]);
                        umma_commit_el(&empty[ks]);
                        if (j == end - 1) umma_commit_el(q_empty);
                        return true;
                    };
                    if (end == u.t0) {
                        umma_commit_el(q_empty);
                    } else if (!next_s(u.t0)) {
                        ok = false;
                        break;
                    }
                    for (int j = u.t0; j < end; ++j) {
                        if (j + 1 < end && !next_s(j + 1)) {  // S of the next tile ahead of PV
                            ok = false;
                            break;
                        }
                        const int x = n + 2 * (j - u.t0) + 1, vs = x % L::kSlots;
                        const int gg = g + j - u.t0;
                        if (!mbar_wait_warp(&full[vs], (x / L::kSlots) & 1, p.ctl, abort_flag)) {
                            ok = false;
                            break;
                        }
                        clear_tail(u.len, j, vs);
                        if (!mbar_wait_warp(&p_full[gg & 1], (gg >> 1) & 1, p.ctl, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        issue_pv(0, gg & 1, vs, j > u.t0);
                        umma_commit_el(pv_done);
                        umma_commit_el(&empty[vs]);
                    }
                    if (!ok) break;
                    n += 2 * (end - u.t0);
                    g += end - u.t0;
                    if (end > u.t0) umma_commit_el(&o_final[0]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&unit_empty[e]);
            }
            // every MMA issued above completes before the CTA releases TMEM and smem
            umma_commit_el(drain);
            drain_wait(drain, 0, p.ctl);
            __syncwarp();
        }
    } else {
        if constexpr (TILES == 2) regs_inc<208>();
        // ---------------------------------------------------------------- softmax warps
        using T = elem_t<BF16>;
        const int t = TILES == 2 ? (warp - L::kSoftWarp) >> 2 : 0;  // query tile
        const int quad = warp & 3;  // a warp may touch TMEM lanes [32*(warp%4), +32)
        const int row = quad * 32 + lane;
        const int row_tok = t * p.tile_toks + row / p.rep, row_head = row % p.rep;
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tO = tmem + lane_base + 256 + t * D;
        const float sl2 = p.scale_log2;
        int scnt = 0;  // score tiles consumed
        int nfin = 0;  // pieces with products (o_final phases)
        for (int k = 0;; ++k) {
            const int e = k & 1;
            if (!mbar_wait_warp(&unit_full[e], (k >> 1) & 1, p.ctl, abort_flag)) break;
            const PieceSlot u = read_slot(e);
            if (u.tok0 < 0) break;
            const int end = piece_end(u, t, p.tile_toks, p.causal);
            // a warp with no row of the unit only keeps the barriers going
            const bool real = row_tok < min(u.toks, (t + 1) * p.tile_toks);
            const bool busy = __any_sync(0xffffffffu, real);
            const int last = u.last0 + (p.causal ? row_tok : 0);  // last key this row sees
            float m = -INFINITY;  // running (reference) max of the scaled scores, log2 units
            float l = 0.f;        // running sum of exp2(score - m)
            bool ok = true;
            for (int j = u.t0; j < end; ++j, ++scnt) {
                const int buf = TILES == 2 ? t : (scnt & 1);
                const uint32_t par = TILES == 2 ? (scnt & 1) : ((scnt >> 1) & 1);
                if (!mbar_wait_warp(&s_full[buf], par, p.ctl, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (busy) {
                    const uint32_t tS = tmem + lane_base + buf * 128;
                    uint32_t r[128];
                    tmem_ld32(tS + 0, r + 0);
                    tmem_ld32(tS + 32, r + 32);
                    tmem_ld32(tS + 64, r + 64);
                    tmem_ld32(tS + 96, r + 96);
                    tmem_wait_ld();
                    const int lim = last - j * kPagedKeys;  // columns above lim are masked
                    if (lim < kPagedKeys - 1) {
#pragma unroll
                        for (int c = 0; c < 128; ++c)
                            if (c > lim) r[c] = __float_as_uint(-INFINITY);
                    }
                    const float m_tile = row_max128(r) * sl2;
                    const float m_new = fmaxf(m, m_tile);
                    const bool old_finite = m != -INFINITY;
                    const bool grow = m_new > m + 8.0f;
                    float alpha = 1.f;
                    if (grow) {
                        if (old_finite) alpha = ex2(m - m_new);
                        l *= alpha;
                        m = m_new;
                    }
                    const bool rescale = grow && old_finite;
                    const float mu = m == -INFINITY ? 0.f : m;  // nothing unmasked yet
                    float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                     make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    const float2 sc2 = make_float2(sl2, sl2), mu2 = make_float2(-mu, -mu);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // the probabilities are rounded to the inputs' type for the product (its
                        // operand has 16 bits); their sum keeps the fp32 ones
                        uint32_t pk[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float2 x =
                                ffma2(make_float2(__uint_as_float(r[64 * h + 2 * c]),
                                                  __uint_as_float(r[64 * h + 2 * c + 1])),
                                      sc2, mu2);
                            const float2 ev = make_float2(ex2(x.x), ex2(x.y));
                            acc[c & 3] = fadd2(acc[c & 3], ev);
                            pk[c] = pack2<BF16>(ev.x, ev.y);
                        }
                        tmem_st32(tS + 32 * h, pk);
                    }
                    const float2 a01 = fadd2(acc[0], acc[1]), a23 = fadd2(acc[2], acc[3]);
                    const float2 a = fadd2(a01, a23);
                    l += a.x + a.y;
                    if (__any_sync(0xffffffffu, rescale)) {
                        // two tiles: the previous PV into O_t completed before this S_t; one
                        // tile: S was issued ahead of it, so wait for it
                        if constexpr (TILES == 1) {
                            if (!mbar_wait_warp(pv_done, (scnt - 1) & 1, p.ctl, abort_flag)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                        }
#pragma unroll
                        for (int cc = 0; cc < D / 32; ++cc) {
                            uint32_t o[32];
                            tmem_ld32(tO + cc * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                            tmem_st32(tO + cc * 32, o);
                        }
                    }
                }
                mbar_arrive_warp_after_st(&p_full[buf]);
            }
            if (!ok) break;
            if (end > u.t0) {
                if (!mbar_wait_warp(&o_final[t], nfin & 1, p.ctl, abort_flag)) break;
                ++nfin;
                tc_fence_after();
            }
            if (busy) {
                // O and LSE, or the piece's partial (m, l, O~); the tensor-memory loads are
                // warp-wide, the stores only for real rows
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const int head = u.kvh * p.rep + row_head;
                const long tok = u.tok0 + row_tok;
                const long prow = static_cast<long>(u.dest) * p.part_rows + t * 128 + row;
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    if (end > u.t0) {
                        tmem_ld32(tO + cc * 32, o);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = 0u;
                    }
                    if (!real) continue;
                    if (u.dest < 0) {
                        uint4 *dst = reinterpret_cast<uint4 *>(
                            reinterpret_cast<T *>(p.o) + tok * p.o_t + head * p.o_h + cc * 32);
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4) {
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                w[x] = pack2<BF16>(__uint_as_float(o[8 * q4 + 2 * x]) * inv,
                                                   __uint_as_float(o[8 * q4 + 2 * x + 1]) * inv);
                            dst[q4] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(p.part_o + prow * D + cc * 32);
#pragma unroll
                        for (int q4 = 0; q4 < 8; ++q4)
                            dst[q4] = make_float4(
                                __uint_as_float(o[4 * q4]), __uint_as_float(o[4 * q4 + 1]),
                                __uint_as_float(o[4 * q4 + 2]), __uint_as_float(o[4 * q4 + 3]));
                    }
                }
                if (real) {
                    if (u.dest < 0)
                        p.lse[tok * p.c.H + head] = row_lse(m, l);
                    else
                        p.part_ml[prow] = make_float2(m, l);
                }
            }
            // O has been read out (the next unit's first PV waits for this warp's next p_full
            // arrival); the unit slot is no longer needed
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&unit_empty[e]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Merge of the units that borders cut: block c does the unit whose first piece CTA c ended with,
// one row per warp.  The pieces stand in CTA order: M = max m_s, w_s = 2^(m_s - M), l = sum w_s l_s,
// O = sum w_s O_s / l, LSE = (M + log2 l) ln 2, in that order (deterministic).
constexpr int kMergeWarps = 4;
template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeWarps * 32) fa_paged_merge_kernel(const PagedAttnParams p) {
    using T = elem_t<BF16>;
    constexpr int kCols = D / 32;
    constexpr int kBatch = 8;  // pieces whose partial outputs are in flight at once
    griddep_wait();
    const int c = static_cast<int>(blockIdx.x), lane = lane_id();
    const int4 cut = p.cut[2 * c];
    const int pieces = p.cut[2 * c + 1].x;
    if (pieces < 2) return;
    const int tok0 = cut.x, toks = cut.y, kvh = cut.z;
    auto slot = [&](int s) { return static_cast<long>(s == 0 ? 2 * c + 1 : 2 * (c + s)); };
    for (int r = blockIdx.y * kMergeWarps + warp_id(); r < p.part_rows;
         r += gridDim.y * kMergeWarps) {
        const int t = r >> 7, row = r & 127;
        const int tok = t * p.tile_toks + row / p.rep;
        if (row >= p.tile_toks * p.rep || tok >= toks) continue;
        float M = -INFINITY;
        for (int s = lane; s < pieces; s += 32) M = fmaxf(M, p.part_ml[slot(s) * p.part_rows + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float l = 0.f, acc[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
        for (int s0 = 0; s0 < pieces; s0 += kBatch) {
            float2 ml[kBatch];
            float x[kBatch][kCols];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const long pr = slot(min(s0 + i, pieces - 1)) * p.part_rows + r;
                ml[i] = p.part_ml[pr];
#pragma unroll
                for (int e = 0; e < kCols; ++e) x[i][e] = p.part_o[pr * D + lane * kCols + e];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                // a piece that saw nothing (l = 0) weighs nothing; one whose scores are all NaN
                // (m = -inf, l = NaN) passes its NaN on
                if (s0 + i >= pieces || ml[i].y == 0.f) continue;
                const float w = ml[i].x == -INFINITY ? 1.f : ex2(ml[i].x - M);
                l = fmaf(w, ml[i].y, l);
#pragma unroll
                for (int e = 0; e < kCols; ++e) acc[e] = fmaf(w, x[i][e], acc[e]);
            }
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int head = kvh * p.rep + row % p.rep;
        T *dst = reinterpret_cast<T *>(p.o) + static_cast<long>(tok0 + tok) * p.o_t + head * p.o_h +
                 lane * kCols;
#pragma unroll
        for (int e = 0; e < kCols; e += 2)
            reinterpret_cast<uint32_t *>(dst + e)[0] = pack2<BF16>(acc[e] * inv, acc[e + 1] * inv);
        if (lane == 0)
            p.lse[static_cast<long>(tok0 + tok) * p.c.H + head] = row_lse(M, l);
    }
}

template <int D, bool BF16, int TILES>
cudaError_t launch_attn_t(const PagedMaps &m, const PagedAttnParams &p, cudaStream_t stream) {
    using L = PagedLayout<D, TILES>;
    auto kern = fa_paged_attn_kernel<D, BF16, TILES>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
    if (e != cudaSuccess) return e;
    kern<<<kPagedCtas, L::kThreads, L::kAlloc, stream>>>(m, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.cut == nullptr) return e;
    cudaLaunchConfig_t cfg = {};
    const int rows = p.part_rows;  // about four rows per warp, and few blocks where rows are few
    cfg.gridDim = dim3(kPagedCtas - 1, (rows + 4 * kMergeWarps - 1) / (4 * kMergeWarps));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa_paged_merge_kernel<D, BF16>, p);
}

template <int D, bool BF16>
cudaError_t launch_attn_d(const PagedMaps &m, const PagedAttnParams &p, int tiles,
                          cudaStream_t st) {
    return tiles == 2 ? launch_attn_t<D, BF16, 2>(m, p, st) : launch_attn_t<D, BF16, 1>(m, p, st);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedMaps &m, const PagedAttnParams &p, int d, bool bf16,
                              int tiles, cudaStream_t stream) {
    if (d == 64) return bf16 ? launch_attn_d<64, true>(m, p, tiles, stream)
                             : launch_attn_d<64, false>(m, p, tiles, stream);
    return bf16 ? launch_attn_d<128, true>(m, p, tiles, stream)
                : launch_attn_d<128, false>(m, p, tiles, stream);
}

}  // namespace fa
