// fa_paged_attn.cu - attention of the new tokens of every sequence over its paged cache, sm_103a.
//
// Row i of the n new tokens of sequence b sees the keys j <= kv_len[b] - n + i (causal) or all
// kv_len[b] of them: O = softmax(scale q K^T) V and the logsumexp, by the online softmax
// (FlashAttention-2 reading notes, Algorithm 1) with the statistic merge of the FlashAttention
// paper detail, Technique 1, for units whose keys are spread over several CTAs.
//
// Rows.  The query heads of a K/V head's group share its keys, so a query tile of 128 rows is
// floor(128 / rep) tokens times the rep heads of one group: one TMA box of the token-major Q.  A
// prompt chunk's unit is two such tiles, one for each of the two softmax groups, which share every
// K/V tile (256 rows per tile read from L2, as in the forward).  A unit of no more tokens than one
// tile (single tokens, drafted ones) gives both groups the same query tile and alternate key
// tiles: the chain from a score tile to its probabilities takes longer than HBM needs to bring the
// next tile, and two of them in flight hide it.  At the end the second group's statistics and
// accumulator (the same tensor-memory lanes) are merged into the first's.
//
// Keys.  A tile is 128 positions, whatever the page size: its pages are loaded by one TMA box each
// into their rows of the 128-byte-swizzled tile (a page of 8 rows or more starts on a swizzle
// atom); pages behind the sequence's end are loaded from an index outside the pool, which TMA
// fills with zeros.  Scores behind the end are masked, and V's rows between the end and the end of
// its page are zeroed in shared memory before the product, so that whatever the cache holds there
// (NaN included) meets a probability of zero as a zero.  K and V have a ring and a load warp each:
// a page of 16 rows is a box of 2 KB, and one warp alone issued them no faster than 5.6 TB/s.
//
// Work.  paged.cuh cuts the line of all units' key tiles into one equal stretch per CTA, on the
// device (the host knows no lengths), so prompt chunks and single tokens of any mixture balance,
// and a single sequence's keys spread over all SMs.
//
// Warps: 0 walks the units and loads Q and K, 2 loads V, 1 issues the MMAs, 4..7 and 8..11 are the
// softmax groups.  MMA order per step: PV_0 of the step before, S_0, PV_1, S_1, as in the forward.
#include "paged.cuh"

#include <type_traits>

namespace fa {
namespace {

// QT: query tiles that a unit may have (1: no sequence brings more tokens than one tile holds).
template <int D, int QT>
struct PagedLayout {
    static constexpr int kTileBytes = 128 * D * 2;  // one 128 x d tile of 16-bit values
    static constexpr int kBoxes = D / 64;
    static constexpr int kBoxBytes = 128 * 128;
    // K waits only for its S, V for the softmax: with an odd number of slots V gets the more
    static constexpr int kKSlots = D == 128 ? (QT == 2 ? 2 : 3) : 6;
    static constexpr int kVSlots = D == 128 ? 3 : 6;
    static constexpr int kKOff = QT * kTileBytes;  // after the Q tiles
    static constexpr int kVOff = kKOff + kKSlots * kTileBytes;
    static constexpr int kBarOff = kVOff + kVSlots * kTileBytes;
    // q_full, q_empty, k_full[], k_empty[], v_full[], v_empty[], s_full[2], p_full[2], o_final[2],
    // pair_full, pair_read, unit_full[2], unit_empty[2], drain
    static constexpr int kNumBars = 2 + 2 * kKSlots + 2 * kVSlots + 13;
    static constexpr int kUnitOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;  // two unit slots
    static constexpr int kScanOff = kUnitOff + 2 * 48;  // the plan's sums: 16 longs
    static constexpr int kMiscOff = kScanOff + 16 * 8;  // TMEM base, abort flag
    static constexpr int kPairOff = kMiscOff + 8;       // the second group's (m, l): float2[128]
    static constexpr int kBytes = kPairOff + 128 * 8;
    static constexpr int kAlloc = kBytes + 1024;
    static constexpr int kThreads = 384;
    static constexpr uint32_t kTmemCols = 512;  // S_0, S_1 (2 x 128), O_0, O_1 (2 x d)
    static_assert(kAlloc <= 232448, "shared memory per CTA");
};

template <bool BF16>
using elem_t = typename std::conditional<BF16, __nv_bfloat16, __half>::type;

// Natural logsumexp of a row from its max (log2 units) and sum; a sum that is NaN stays one.
__device__ __forceinline__ float row_lse(float m, float l) {
    if (l == 0.f) return -INFINITY;
    return l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : l;
}

// A unit's piece as the first load warp hands it to the others (one of two slots in shared memory).
struct PieceSlot {
    int tok0;   // first token, in the batch; -1: no more pieces
    int toks;
    int kvh;
    int last0;  // last key that the first token sees
    int len;
    int t0, t1; // key tiles, t1 not beyond what the unit sees
    int dest;   // -1: O and LSE, otherwise the slot of its partial result
    int b;      // sequence
};

// First key tile from t0 on that query tile q of the piece does not take part in.
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
    r.ctas = paged_ctas(r.total, static_cast<int>(gridDim.x));
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

// Page ids of a piece's key tiles for one load warp: 32 at a time in the lanes, the next 32 read
// ahead.  Lane i of a tile's call gets the id of the tile's i-th page; pages behind the sequence's
// end and ids that are no page of the pool come back as num_pages, outside the pool.
struct PageWindow {
    const int *row;
    int have;  // pages of the sequence
    int base, now, next;
    __device__ __forceinline__ int read(const PagedView &c, int first) const {
        const int i = first + lane_id();
        return i < have ? row[i] : c.num_pages;
    }
    __device__ __forceinline__ void open(const PagedView &c, const PieceSlot &u) {
        row = c.table + static_cast<long>(u.b) * c.max_pages;
        have = (u.len + (1 << c.page_shift) - 1) >> c.page_shift;
        base = ((u.t0 * kPagedKeys) >> c.page_shift) & ~31;
        now = read(c, base);
        next = read(c, base + 32);
    }
    __device__ __forceinline__ int tile(const PagedView &c, int j, int boxes) {
        const int page0 = (j * kPagedKeys) >> c.page_shift;
        if (page0 >= base + 32) {
            base += 32;
            now = next;
            next = read(c, base + 32);
        }
        const int i = page0 + lane_id();
        int id = __shfl_sync(0xffffffffu, now, (i - base) & 31);
        if (lane_id() < boxes && i < have && (id < 0 || id >= c.num_pages)) {
            paged_report(c);
            id = c.num_pages;
        }
        return id;
    }
};

template <int D, bool BF16, int QT>
__global__ void __launch_bounds__(384, 1)
    fa_paged_attn_kernel(const __grid_constant__ PagedMaps maps, const PagedAttnParams p) {
    using L = PagedLayout<D, QT>;
    constexpr uint32_t kIdescS = idesc_f16(128, 128, BF16, false);
    constexpr uint32_t kIdescPV = idesc_f16(128, D, BF16, true);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *q_full = bars, *q_empty = bars + 1;
    uint64_t *k_full = bars + 2, *k_empty = k_full + L::kKSlots;
    uint64_t *v_full = k_empty + L::kKSlots, *v_empty = v_full + L::kVSlots;
    uint64_t *s_full = v_empty + L::kVSlots;  // [2]: per softmax group, as the next three
    uint64_t *p_full = s_full + 2;
    uint64_t *o_final = p_full + 2;
    uint64_t *pair_full = o_final + 2, *pair_read = pair_full + 1;
    uint64_t *unit_full = pair_read + 1, *unit_empty = unit_full + 2;  // [2]: per unit slot
    uint64_t *drain = unit_empty + 2;
    volatile int *unit_slot = reinterpret_cast<volatile int *>(smem + L::kUnitOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMiscOff + 4);
    float2 *pair_ml = reinterpret_cast<float2 *>(smem + L::kPairOff);
    const int warp = warp_id(), lane = lane_id();
    const PagedWork work = {p.tile_toks, QT * p.tile_toks, paged_unit_cost(QT), p.causal};

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < L::kKSlots; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < L::kVSlots; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);  // one arrival per softmax warp of a group
            mbar_init(&o_final[i], 1);
            mbar_init(&unit_full[i], 1);
            mbar_init(&unit_empty[i], 10);  // the MMA warp, the V warp and the softmax warps
        }
        mbar_init(pair_full, 4);
        mbar_init(pair_read, 4);
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
        volatile int *s = unit_slot + 12 * e;
        u.tok0 = s[0];
        u.toks = s[1];
        u.kvh = s[2];
        u.last0 = s[3];
        u.len = s[4];
        u.t0 = s[5];
        u.t1 = s[6];
        u.dest = s[7];
        u.b = s[8];
        return u;
    };
    // both groups work on the same query tile and take alternate key tiles
    auto is_pair = [&](const PieceSlot &u) { return QT == 1 || u.toks <= p.tile_toks; };

    if (warp < 4) {
        // warpgroup 0 gives registers to the softmax groups: 128 x 80 + 256 x 208 = 63488 of the
        // 384 x 168 = 64512 the CTA is launched with
        regs_dec<80>();
        const int box_rows = min(1 << p.c.page_shift, kPagedKeys);  // rows of one page in a tile
        const int boxes = kPagedKeys / box_rows;                    // pages of a tile
        // key tile j's pages from K's or V's map into a ring slot: one lane per page
        auto load_tile = [&](const CUtensorMap *map, const PieceSlot &u, int j, int id,
                             uint8_t *slot, uint64_t *bar) {
            if (lane == 0) mbar_arrive_expect_tx(bar, L::kTileBytes);
            __syncwarp();
            if (lane < boxes) {
                const int y = (j * kPagedKeys) & ((1 << p.c.page_shift) - 1);
                uint8_t *dst = slot + lane * box_rows * 128;
                for (int b = 0; b < L::kBoxes; ++b)
                    tma_load_4d(dst + b * L::kBoxBytes, map, b * 64, maps.rows_inner ? y : u.kvh,
                                maps.rows_inner ? u.kvh : y, id, bar);
            }
        };
        if (warp == 0) {
            // ------------------------------------------------- units, Q and K
            int n = 0;   // K tiles issued
            int nq = 0;  // Q loads issued
            int k = 0;   // pieces so far
            bool ok = true;
            PagedCursor cur;
            long room = mine.end - mine.begin;
            if (room > 0) cur.start(p.c, work, mine.seq, mine.begin - mine.before);
            int4 cut0 = make_int4(-1, 0, 0, 0);  // what the merge has to do for this CTA
            int cut_n = 0;
            for (;;) {
                PieceSlot u;
                u.tok0 = -1;
                while (room > 0) {
                    const long at = mine.end - room;
                    const PagedPiece x = cur.take(p.c, work, room);
                    if (x.t0 == x.t1) continue;
                    const bool whole = x.t1 - x.t0 == x.tiles;
                    if (!whole && x.t0 == 0) {  // starts a unit that other CTAs finish
                        const long end = at + x.unit_end;
                        cut0 = make_int4(x.tok0, x.toks, x.kvh, 0);
                        cut_n = static_cast<int>((end * mine.ctas + mine.total - 1) / mine.total) -
                                static_cast<int>(blockIdx.x);
                    }
                    u.tok0 = x.tok0;
                    u.toks = x.toks;
                    u.kvh = x.kvh;
                    u.last0 = x.last0;
                    u.len = x.len;
                    u.t0 = x.t0;
                    // a unit that stands before its sequence sees nothing
                    u.t1 = x.last0 + (p.causal ? x.toks - 1 : 0) < 0 ? x.t0 : x.t1;
                    u.dest = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (x.t0 == 0 ? 1 : 0);
                    u.b = x.b;
                    break;
                }
                const int e = k & 1;
                if (k >= 2 && !mbar_wait_warp(&unit_empty[e], ((k >> 1) - 1) & 1, p.ctl,
                                              abort_flag)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    volatile int *s = unit_slot + 12 * e;
                    s[0] = u.tok0;
                    if (u.tok0 >= 0) {
                        s[1] = u.toks;
                        s[2] = u.kvh;
                        s[3] = u.last0;
                        s[4] = u.len;
                        s[5] = u.t0;
                        s[6] = u.t1;
                        s[7] = u.dest;
                        s[8] = u.b;
                    }
                    mbar_arrive(&unit_full[e]);
                }
                __syncwarp();
                if (u.tok0 < 0) break;
                ++k;
                PageWindow win;
                win.open(p.c, u);
                auto load_q = [&]() {  // the Q tiles are free once the last unit's last S is done
                    if (nq > 0 && !mbar_wait_warp(q_empty, (nq - 1) & 1, p.ctl, abort_flag))
                        return false;
                    if (lane == 0) {
                        const int tiles = is_pair(u) ? 1 : 2;
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
                bool q_done = false;
                if (nq == 0) ok = q_done = load_q();  // the first Q needs no page id
                for (int j = u.t0; j < u.t1 && ok; ++j) {
                    const int id = win.tile(p.c, j, boxes), s = n % L::kKSlots;
                    if (!mbar_wait_warp(&k_empty[s], ((n / L::kKSlots) & 1) ^ 1, p.ctl,
                                        abort_flag)) {
                        ok = false;
                        break;
                    }
                    load_tile(&maps.k, u, j, id, smem + L::kKOff + s * L::kTileBytes, &k_full[s]);
                    ++n;
                    // the first K goes ahead of Q: its slot frees before the Q tiles do
                    if (!q_done) {
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
                    for (int l = n > L::kKSlots ? n - L::kKSlots : 0; l < n; ++l)
                        drain_wait(&k_full[l % L::kKSlots], (l / L::kKSlots) & 1, p.ctl);
                }
            }
            __syncwarp();
        } else if (warp == 2) {
            // ------------------------------------------------- V
            int n = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int e = k & 1;
                if (!mbar_wait_warp(&unit_full[e], (k >> 1) & 1, p.ctl, abort_flag)) {
                    ok = false;
                    break;
                }
                const PieceSlot u = read_slot(e);
                if (u.tok0 < 0) break;
                PageWindow win;
                win.open(p.c, u);
                for (int j = u.t0; j < u.t1; ++j) {
                    const int id = win.tile(p.c, j, boxes), s = n % L::kVSlots;
                    if (!mbar_wait_warp(&v_empty[s], ((n / L::kVSlots) & 1) ^ 1, p.ctl,
                                        abort_flag)) {
                        ok = false;
                        break;
                    }
                    load_tile(&maps.v, u, j, id, smem + L::kVOff + s * L::kTileBytes, &v_full[s]);
                    ++n;
                }
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&unit_empty[e]);
            }
            if (!ok || *abort_flag) {
                if (lane == 0)
                    for (int l = n > L::kVSlots ? n - L::kVSlots : 0; l < n; ++l)
                        drain_wait(&v_full[l % L::kVSlots], (l / L::kVSlots) & 1, p.ctl);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------- MMA issuer
            const SDesc dq0 = sdesc_make(smem_u32(smem), 16, 1024);              // Q: K-major
            const SDesc dk0 = sdesc_make(smem_u32(smem + L::kKOff), 16, 1024);   // K: K-major
            const SDesc dv0 = sdesc_make(smem_u32(smem + L::kVOff), L::kBoxBytes,
                                         1024);                                   // V: MN-major
            auto issue_s = [&](int q, int t, int ks) {
                const SDesc a = sdesc_add(dq0, q * L::kTileBytes);
                const SDesc b = sdesc_add(dk0, ks * L::kTileBytes);
                if constexpr (D == 128)
                    mma_ss_chain_k128(tmem + t * 128, a, b, kIdescS, 0u);
                else
                    mma_ss_chain_k64(tmem + t * 128, a, b, kIdescS, 0u);
                umma_commit_el(&s_full[t]);
            };
            auto issue_pv = [&](int t, int vs, bool accumulate) {
                mma_ts_chain_k128(tmem + 256 + t * D, tmem + t * 128,
                                  sdesc_add(dv0, vs * L::kTileBytes), kIdescPV,
                                  accumulate ? 1u : 0u);
            };
            auto wait_k = [&](int x) {
                if (!mbar_wait_warp(&k_full[x % L::kKSlots], (x / L::kKSlots) & 1, p.ctl,
                                    abort_flag))
                    return false;
                tc_fence_after();
                return true;
            };
            // V tile x of the ring (key tile j) has landed; its rows from the sequence's end to
            // the end of that page become zeros (pages behind it were loaded as zeros)
            auto wait_v = [&](int x, int j, int len) {
                const int vs = x % L::kVSlots;
                if (!mbar_wait_warp(&v_full[vs], (x / L::kVSlots) & 1, p.ctl, abort_flag))
                    return false;
                const int r0 = len - j * kPagedKeys;
                if (r0 < kPagedKeys) {
                    const int size = 1 << p.c.page_shift;
                    const int r1 = min(kPagedKeys, (r0 + size - 1) & ~(size - 1));
                    uint8_t *tile = smem + L::kVOff + vs * L::kTileBytes;
                    for (int b = 0; b < L::kBoxes; ++b)
                        for (int a = r0 * 128 + lane * 16; a < r1 * 128; a += 512)
                            *reinterpret_cast<uint4 *>(tile + b * L::kBoxBytes + a) =
                                make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                return true;
            };
            int nt = 0;            // K and V tiles consumed
            int pcnt[2] = {0, 0};  // PV products per group (p_full phases)
            auto wait_p = [&](int t) {
                if (!mbar_wait_warp(&p_full[t], pcnt[t] & 1, p.ctl, abort_flag)) return false;
                tc_fence_after();
                return true;
            };
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
                const int p0[2] = {pcnt[0], pcnt[1]};
                const int n0 = nt - u.t0;  // ring index of key tile j is n0 + j
                if (u.t1 == u.t0) umma_commit_el(q_empty);  // nothing seen: Q is free at once
                if (is_pair(u)) {
                    // step by step, group t takes tile j + t
                    for (int j = u.t0; ok && j - 2 < u.t1; j += 2) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int jp = j + t - 2, jn = j + t;
                            if (jp >= u.t0 && jp < u.t1) {
                                if (!wait_v(n0 + jp, jp, u.len) || !wait_p(t)) {
                                    ok = false;
                                    break;
                                }
                                issue_pv(t, (n0 + jp) % L::kVSlots, pcnt[t] > p0[t]);
                                ++pcnt[t];
                                umma_commit_el(&v_empty[(n0 + jp) % L::kVSlots]);
                            }
                            if (jn < u.t1) {
                                if (!wait_k(n0 + jn)) {
                                    ok = false;
                                    break;
                                }
                                issue_s(0, t, (n0 + jn) % L::kKSlots);
                                umma_commit_el(&k_empty[(n0 + jn) % L::kKSlots]);
                                if (jn == u.t1 - 1) umma_commit_el(q_empty);
                            }
                        }
                    }
                } else {
                    // both groups take every tile, group t for query tile t
                    const int end[2] = {piece_end(u, 0, p.tile_toks, p.causal),
                                        piece_end(u, 1, p.tile_toks, p.causal)};
                    for (int j = u.t0; ok && j <= u.t1; ++j) {
                        const int vs = (n0 + j - 1 + L::kVSlots) % L::kVSlots;
                        if (j < u.t1 && !wait_k(n0 + j)) {
                            ok = false;
                            break;
                        }
                        bool v_ready = false;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (j > u.t0 && j - 1 < end[t]) {
                                if (!v_ready && !wait_v(n0 + j - 1, j - 1, u.len)) {
                                    ok = false;
                                    break;
                                }
                                v_ready = true;
                                if (!wait_p(t)) {
                                    ok = false;
                                    break;
                                }
                                issue_pv(t, vs, pcnt[t] > p0[t]);
                                ++pcnt[t];
                            }
                            if (j < end[t]) issue_s(t, t, (n0 + j) % L::kKSlots);
                        }
                        if (!ok) break;
                        if (j == u.t1 - 1) umma_commit_el(q_empty);
                        if (j > u.t0) umma_commit_el(&v_empty[vs]);
                        if (j < u.t1) umma_commit_el(&k_empty[(n0 + j) % L::kKSlots]);
                    }
                }
                if (!ok) break;
                nt += u.t1 - u.t0;
                // O_t of this piece is final (nobody waits for a group that had no tile)
                for (int t = 0; t < 2; ++t)
                    if (pcnt[t] > p0[t]) umma_commit_el(&o_final[t]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&unit_empty[e]);
            }
            // every MMA issued above completes before the CTA releases TMEM and smem
            umma_commit_el(drain);
            drain_wait(drain, 0, p.ctl);
            __syncwarp();
        }
    } else {
        regs_inc<208>();
        // ---------------------------------------------------------------- softmax groups
        using T = elem_t<BF16>;
        const int t = (warp - 4) >> 2;  // group
        const int quad = warp & 3;      // a warp may touch TMEM lanes [32*(warp%4), +32)
        const int row = quad * 32 + lane;
        const int row_tok = row / p.rep, row_head = row % p.rep;  // within a query tile
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tS = tmem + lane_base + t * 128;
        const uint32_t tO = tmem + lane_base + 256 + t * D;
        const float sl2 = p.scale_log2;
        int scnt = 0;          // score tiles consumed by this group
        int nfin = 0;          // pieces in which this group had products (o_final phases)
        int nfin1 = 0;         // first group: the same of the second
        int npair = 0;         // merges between the groups (pair_full, pair_read phases)
        bool owed = false;     // second group: the first has still to read what it left
        for (int k = 0;; ++k) {
            const int e = k & 1;
            if (!mbar_wait_warp(&unit_full[e], (k >> 1) & 1, p.ctl, abort_flag)) break;
            const PieceSlot u = read_slot(e);
            if (u.tok0 < 0) break;
            const bool pair = is_pair(u);
            const int q = pair ? 0 : t;  // query tile
            const int first = u.t0 + (pair ? t : 0), step = pair ? 2 : 1;
            const int end = pair ? u.t1 : piece_end(u, t, p.tile_toks, p.causal);
            // a warp with no row of the unit only keeps the barriers going
            const int tok = q * p.tile_toks + row_tok;
            const bool real = row_tok < p.tile_toks && tok < u.toks;
            const bool busy = __any_sync(0xffffffffu, real);
            const int last = u.last0 + (p.causal ? tok : 0);  // last key this row sees
            float m = -INFINITY;  // running (reference) max of the scaled scores, log2 units
            float l = 0.f;        // running sum of exp2(score - m)
            bool ok = true;
            for (int j = first; j < end; j += step) {
                if (!mbar_wait_warp(&s_full[t], scnt & 1, p.ctl, abort_flag)) {
                    ok = false;
                    break;
                }
                ++scnt;
                tc_fence_after();
                if (busy) {
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
                        // the previous PV into O_t completed before this S_t, and the next one
                        // waits for p_full, so O_t is ours to rescale
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
                if (owed) {  // this arrival lets the next PV overwrite what was left in O_1
                    if (!mbar_wait_warp(pair_read, (npair - 1) & 1, p.ctl, abort_flag)) {
                        ok = false;
                        break;
                    }
                    owed = false;
                }
                mbar_arrive_warp_after_st(&p_full[t]);
            }
            if (!ok) break;
            const bool had = first < end;
            const bool both = pair && u.t1 - u.t0 > 1;  // the second group has a share
            if (t == 1 && pair) {
                if (both) {  // its statistics for the first group, which finds O_1 in place
                    pair_ml[row] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pair_full);
                    ++npair;
                    ++nfin;
                    owed = true;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&unit_empty[e]);
                continue;
            }
            if (had) {
                if (!mbar_wait_warp(&o_final[t], nfin & 1, p.ctl, abort_flag)) break;
                ++nfin;
            }
            float wa = 1.f, wb = 0.f;  // weights of O_0 and of the second group's O_1
            if (both) {
                if (!mbar_wait_warp(pair_full, npair & 1, p.ctl, abort_flag)) break;
                if (!mbar_wait_warp(&o_final[1], nfin1 & 1, p.ctl, abort_flag)) break;
                ++npair;
                ++nfin1;
                const float2 o = pair_ml[row];
                const float M = fmaxf(m, o.x), mu = M == -INFINITY ? 0.f : M;
                wa = ex2(m - mu);
                wb = ex2(o.x - mu);
                l = l * wa + o.y * wb;
                m = M;
            } else if (t == 0 && !pair && piece_end(u, 1, p.tile_toks, p.causal) > u.t0) {
                ++nfin1;  // the second group waits for its own
            }
            tc_fence_after();
            if (busy) {
                // O and LSE, or the piece's partial (m, l, O~); the tensor-memory loads are
                // warp-wide, the stores only for real rows
                const float inv = u.dest >= 0 ? 1.f : l > 0.f ? 1.f / l : 0.f;
                wa *= inv;
                wb *= inv;
                const int head = u.kvh * p.rep + row_head;
                const long otok = u.tok0 + tok;
                const long prow = static_cast<long>(u.dest) * p.part_rows + q * 128 + row;
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    if (had) {
                        tmem_ld32(tO + cc * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            o[x] = __float_as_uint(__uint_as_float(o[x]) * wa);
                    } else {
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = 0u;
                    }
                    if (both) {
                        uint32_t o1[32];
                        tmem_ld32(tO + D + cc * 32, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            o[x] = __float_as_uint(
                                fmaf(__uint_as_float(o1[x]), wb, __uint_as_float(o[x])));
                    }
                    if (!real) continue;
                    if (u.dest < 0) {
                        uint4 *dst = reinterpret_cast<uint4 *>(
                            reinterpret_cast<T *>(p.o) + otok * p.o_t + head * p.o_h + cc * 32);
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4) {
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                w[x] = pack2<BF16>(__uint_as_float(o[8 * q4 + 2 * x]),
                                                   __uint_as_float(o[8 * q4 + 2 * x + 1]));
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
                        p.lse[otok * p.c.H + head] = row_lse(m, l);
                    else
                        p.part_ml[prow] = make_float2(m, l);
                }
            }
            // O has been read out (the next unit's first PV into it waits for this warp's next
            // p_full arrival, or the second group's after pair_read)
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (both) mbar_arrive(pair_read);
                mbar_arrive(&unit_empty[e]);
            }
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
// one row per warp at a time.  The pieces stand in CTA order and are folded in in that order
// (deterministic), a batch at a time with all its reads in flight: M = max m_s, w_s = 2^(m_s - M),
// l = sum w_s l_s, O = sum w_s O_s / l, LSE = (M + log2 l) ln 2.
constexpr int kMergeWarps = 8;
template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeWarps * 32) fa_paged_merge_kernel(const PagedAttnParams p) {
    using T = elem_t<BF16>;
    constexpr int kCols = D / 32;
    constexpr int kBatch = 8;
    griddep_wait();
    const int c = static_cast<int>(blockIdx.x), lane = lane_id();
    const int4 cut = p.cut[2 * c];
    const int pieces = p.cut[2 * c + 1].x;
    if (pieces < 2) return;
    const int tok0 = cut.x, toks = cut.y, kvh = cut.z;
    const int r = static_cast<int>(blockIdx.y) * kMergeWarps + warp_id();
    const int row = r & 127, row_tok = row / p.rep, tok = (r >> 7) * p.tile_toks + row_tok;
    if (r >= p.part_rows || row_tok >= p.tile_toks || tok >= toks) return;
    float M = -INFINITY, l = 0.f, acc[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
    for (int s0 = 0; s0 < pieces; s0 += kBatch) {
        float2 ml[kBatch];
        float x[kBatch][kCols];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            ml[i] = make_float2(-INFINITY, 0.f);
            if (s0 + i < pieces) {
                const long slot = s0 + i == 0 ? 2 * c + 1 : 2 * (c + s0 + i);
                const long pr = slot * p.part_rows + r;
                ml[i] = p.part_ml[pr];
#pragma unroll
                for (int e = 0; e < kCols; ++e) x[i][e] = p.part_o[pr * D + lane * kCols + e];
            }
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[i].x);
        const float mu = top == -INFINITY ? 0.f : top;
        const float back = ex2(M - mu);
        M = top;
        l *= back;
#pragma unroll
        for (int e = 0; e < kCols; ++e) acc[e] *= back;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            // a piece that saw nothing (l = 0) weighs nothing; one whose scores are all NaN
            // (m = -inf, l = NaN) passes its NaN on
            if (s0 + i >= pieces || ml[i].y == 0.f) continue;
            const float w = ml[i].x == -INFINITY ? 1.f : ex2(ml[i].x - mu);
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
    if (lane == 0) p.lse[static_cast<long>(tok0 + tok) * p.c.H + head] = row_lse(M, l);
}

template <int D, bool BF16, int QT>
cudaError_t launch_attn_t(const PagedMaps &m, const PagedAttnParams &p, cudaStream_t stream) {
    using L = PagedLayout<D, QT>;
    auto kern = fa_paged_attn_kernel<D, BF16, QT>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
    if (e != cudaSuccess) return e;
    kern<<<kPagedCtas, L::kThreads, L::kAlloc, stream>>>(m, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.cut == nullptr) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPagedCtas - 1, (p.part_rows + kMergeWarps - 1) / kMergeWarps);
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
