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
// next tile, and two of them in flight hide it.  At the end one group's statistics and accumulator
// (the same tensor-memory lanes) are merged into those of the other, which had the first tile.  Where no unit
// has two query tiles the groups go on taking turns from unit to unit and a unit's first scores are
// issued before the last one's products: built, that took 1024 sequences of up to 500 keys from 465 to
// 399 us.
//
// Keys.  A tile is 128 positions, whatever the page size: its pages are loaded by one TMA box each
// into their rows of the 128-byte-swizzled tile (a page of 8 rows or more starts on a swizzle
// atom).  Scores behind the sequence's end are masked, whatever K's rows hold there.  V's pages behind the
// end are loaded from an index outside the pool, which TMA fills with zeros, and its rows between
// the end and the end of its page are zeroed in shared memory before the product, so that whatever
// the cache holds there (NaN included) meets a probability of zero as a zero.  K and V have a ring and a load warp each:
// a page of 16 rows is a box of 2 KB, and one warp alone issued them no faster than 5.6 TB/s.
//
// Work.  paged.cuh cuts the line of all units' key tiles into one equal stretch per CTA, on the
// device (the host knows no lengths), so prompt chunks and single tokens of any mixture balance,
// and a single sequence's keys spread over all SMs.
//
// Few units of few keys (a sequence or two, a short cache) are bound by latency: the cut line and
// the merge in a second grid cost more than they balance.  While every unit fits one cluster and
// all clusters fit the chip at once, a cluster of up to eight CTAs takes a unit, each CTA an equal
// share of its key tiles, and the partial results are merged through distributed shared memory in
// the same launch, with no workspace.
//
// Code.  The loops over key tiles are unrolled, what runs once or a few times a unit is rolled up: with
// short sequences every part of the kernel runs from a cold instruction cache, and fetching it was
// most of the time (1024 sequences of up to 500 keys take 306 us, of up to 100 125; with the epilogue
// alone unrolled 314 and 147).
//
// Warps: 0 walks the units and loads Q and K, 2 loads V, 1 issues the MMAs, 4..7 and 8..11 are the
// softmax groups.  MMA order per step: PV_0 of the step before, S_0, PV_1, S_1, as in the forward.
#include "paged.cuh"

#include <atomic>
#include <type_traits>

namespace fa {
namespace {

// QT: query tiles that a unit may have (1: no sequence brings more tokens than one tile holds).
template <int D, int QT, bool CL>
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
    static constexpr int kUnits = 4;  // unit slots: the loads run up to three units ahead
    // Score buffers in tensor memory, 128 columns each, before O_0 and O_1.  A third one, where it
    // fits, has a group's next scores ready before its last product is issued.  Clusters, bound by the
    // chain of their few tiles, gain (8 x 4 tokens 10.05 -> 9.7 us, 30 x 2 12.2 -> 11.9); the line, whose
    // units end a tile later for it, lost (64 tokens over up to 2000 keys 30.8 -> 31.4).
    static constexpr int kBufs = D == 64 && QT == 1 && CL ? 3 : 2;
    static_assert(kUnits > kBufs, "a unit's last products wait for the units after it");
    static constexpr int kOCol = kBufs * 128;
    // q_full[2], q_empty[2], k_full[], k_empty[], v_full[], v_empty[], s_full[], p_full[],
    // o_final[2], pair_full, pair_read, unit_full[], unit_empty[], drain
    static constexpr int kNumBars =
        4 + 2 * kKSlots + 2 * kVSlots + 2 * kBufs + 4 + 2 * kUnits + 1;
    static constexpr int kUnitOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kMiscOff = kUnitOff + kUnits * 32;  // TMEM base, abort flag
    static constexpr int kPairOff = kMiscOff + 8;       // the second group's (m, l): float2[128]
    static constexpr int kBytes = kPairOff + 128 * 8;
    static constexpr int kAlloc = kBytes + 1024;
    // CL: a row of O~ laid over the rings, padded so that neighbouring rows' pieces fall into
    // different banks
    static constexpr int kRowBytes = (D + 4) * 4;
    static_assert(QT * 128 * kRowBytes <= (kKSlots + kVSlots) * kTileBytes, "O~ over the rings");
    static constexpr int kThreads = 384;
    static constexpr uint32_t kTmemCols = 512;  // the score buffers, O_0, O_1 (2 x d)
    static_assert(kOCol + 2 * D <= 512, "tensor memory");
    static_assert(kAlloc <= 232448, "shared memory per CTA");
};

template <bool BF16>
using elem_t = typename std::conditional<BF16, __nv_bfloat16, __half>::type;

// Natural logsumexp of a row from its max (log2 units) and sum; a sum that is NaN stays one.
__device__ __forceinline__ float row_lse(float m, float l) {
    if (l == 0.f) return -INFINITY;
    return l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : l;
}

// Where units have no more than 64 rows, two of them share the Q tile: rows 64 to 127 of its boxes
// are the second buffer.  A product's rows behind the unit's are whatever stands there, and unused.
constexpr int kQBufBytes = 64 * 128;

// Pieces of no more key tiles than this are softmaxed by the rolled-up code: what runs once or twice and
// then makes place for other code costs its fetch.  1024 sequences of up to 500 keys take 323 us without
// it and 306 with 4 or with 8, of up to 100 145 and 125; a tile of a long piece takes a quarter longer in
// it (16 x 8k at d = 64 50.1 -> 57.3).
constexpr int kShortPiece = 4;

constexpr int kDestCluster = -2;
constexpr unsigned kMaxCluster = 8;  // the portable limit

// A unit's piece as the first load warp hands it to the others (a slot in shared memory).
struct PieceSlot {
    int tok0;   // first token, in the batch; -1: no more pieces
    int toks;
    int kvh;
    int last0;  // last key that the first token sees
    int len;
    int t0, t1; // key tiles, t1 not beyond what the unit sees
    int dest;   // -1: O and LSE, kDestCluster: shared memory, otherwise a partial result's slot
};

// First key tile from t0 on that query tile q of the piece does not take part in.
__device__ __forceinline__ int piece_end(const PieceSlot &u, int q, int tile_toks, int causal) {
    const int toks = min(u.toks - q * tile_toks, tile_toks);
    if (toks <= 0) return u.t0;
    const int last = u.last0 + (causal ? q * tile_toks + toks - 1 : 0);
    const int end = last >= 0 ? last / kPagedKeys + 1 : 0;
    return max(u.t0, min(u.t1, end));
}

// Cluster building blocks (PTX barrier.cluster, mapa, ld.shared::cluster).
__device__ __forceinline__ unsigned cluster_size() {
    unsigned n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {  // every thread of every CTA of the cluster
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, unsigned rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// One warp finds unit number `unit` of the batch (CL), a lane per sequence; false: there are fewer.
__device__ __forceinline__ bool find_unit(const PagedView &c, const PagedWork &w, int unit,
                                          bool report, PagedPiece &own) {
    const int lane = lane_id();
    int before = 0;
    bool found = false;
#pragma unroll 1
    for (int b0 = 0; b0 < c.B; b0 += 32) {
        PagedSeq s;
        s.tok0 = s.n = s.len = s.ctx = 0;
        if (b0 + lane < c.B) {
            s = paged_seq(c, b0 + lane);
            if (s.bad && report) paged_report(c);
        }
        const int each = paged_units(s, w), x = each * c.Hkv;
        int upto = x;  // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + upto > unit);
        if (past != 0 && !found) {
            found = true;
            const int at = __ffs(static_cast<int>(past)) - 1;
            const int pos = unit - before - __shfl_sync(0xffffffffu, upto - x, at);
            const int units = __shfl_sync(0xffffffffu, each, at);
            const int tok0 = __shfl_sync(0xffffffffu, s.tok0, at);
            const int n = __shfl_sync(0xffffffffu, s.n, at);
            own.b = b0 + at;
            own.len = __shfl_sync(0xffffffffu, s.len, at);
            own.kvh = pos / units;
            const int i0 = (pos - own.kvh * units) * w.unit_toks;
            own.tok0 = tok0 + i0;
            own.toks = min(n - i0, w.unit_toks);
            const int ctx = __shfl_sync(0xffffffffu, s.ctx, at);
            own.last0 = w.causal ? ctx + i0 : own.len - 1;
            if (!report) return true;  // block 0 goes on to look at every sequence
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return found;
}

// One warp finds its CTA's stretch of the line: the sequences are dealt out to the lanes in equal
// runs (their numbers come from L1 after a run's first read; 32 at a time over the whole batch, 1024
// sequences took 50000 cycles), the sums cut the line, and the lane with the CTA's border has its run looked
// through by all.  Rolled up so that the code is short: it runs once, from a cold instruction cache.
// Returns what the CTA may take and leaves `cur` at its beginning.
__device__ __forceinline__ long find_stretch(const PagedView &c, const PagedWork &w, bool report,
                                             PagedLine &line, PagedCursor &cur) {
    const int lane = lane_id(), cta = static_cast<int>(blockIdx.x);
    const int run = (c.B - 1) / 32 + 1;
    long length = 0, longest = 0, each = 0;
    int heads = 0;
    PagedSeq s;
    s.tok0 = s.n = s.len = s.ctx = 0;
#pragma unroll 1
    for (int i = 0; i < run && lane * static_cast<long>(run) + i < c.B; ++i) {
        const int b = lane * run + i;
        s = paged_seq(c, b);
        if (s.bad && report) paged_report(c);
        each = paged_head(s, w);
        length += c.Hkv * each;
        longest = max(longest, each);
        heads += each > 0 ? c.Hkv : 0;
    }
    long total = length;
    int all = heads;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    line.cut(total, longest, all, w, static_cast<int>(gridDim.x));
    if (cta >= line.ctas) return 0;
    const long begin = line.border(cta);
    // place on the line: lengths, or units counted
    long x = line.by_unit ? heads : length, before = 0;
    int b0 = 0, end = 1;  // (of the runs: one step)
#pragma unroll 1
    for (bool runs = run > 1;; runs = false) {  // over the runs, then over the sequences of one
#pragma unroll 1
        for (; b0 < end; b0 += 32) {
            if (!runs && run > 1) {
                each = 0;
                if (b0 + lane < end) {
                    s = paged_seq(c, b0 + lane);
                    each = paged_head(s, w);
                }
                x = c.Hkv * (line.by_unit ? (each > 0 ? 1 : 0) : each);
            }
            long upto = x;  // inclusive
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + upto > begin);
            if (past == 0) {
                before += __shfl_sync(0xffffffffu, upto, 31);
                continue;
            }
            const int at = __ffs(static_cast<int>(past)) - 1;
            before += __shfl_sync(0xffffffffu, upto - x, at);
            if (runs) {
                b0 = at * run;
                end = min(b0 + run, c.B);
                break;
            }
            s.tok0 = __shfl_sync(0xffffffffu, s.tok0, at);
            s.n = __shfl_sync(0xffffffffu, s.n, at);
            s.len = __shfl_sync(0xffffffffu, s.len, at);
            s.ctx = __shfl_sync(0xffffffffu, s.ctx, at);
            each = __shfl_sync(0xffffffffu, each, at);
            cur.start(c, w, b0 + at, s, line.by_unit ? 1 : each, begin - before);
            return line.by_unit ? each : line.border(cta + 1) - begin;
        }
        if (!runs) return 0;  // (the border lies in one of them)
    }
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
    __device__ __forceinline__ void open(const PagedView &c, const PagedPiece &u) {
        row = c.table + static_cast<long>(u.b) * c.max_pages;
        have = (u.len + (1 << c.page_shift) - 1) >> c.page_shift;
        base = ((u.t0 * kPagedKeys) >> c.page_shift) & ~31;
        now = read(c, base);
        next = read(c, base + 32);
    }
    // pages of the sequence from tile j on
    __device__ __forceinline__ int left(const PagedView &c, int j) const {
        return have - ((j * kPagedKeys) >> c.page_shift);
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

// CL: one unit per cluster, its partial results merged in the cluster.
template <int D, bool BF16, int QT, bool CL>
__global__ void __launch_bounds__(384, 1)
    fa_paged_attn_kernel(const __grid_constant__ PagedMaps maps, const PagedAttnParams p) {
    using L = PagedLayout<D, QT, CL>;
    constexpr uint32_t kIdescS = idesc_f16(128, 128, BF16, false);
    constexpr uint32_t kIdescPV = idesc_f16(128, D, BF16, true);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *q_full = bars, *q_empty = bars + 2;  // [2]: per Q buffer
    uint64_t *k_full = bars + 4, *k_empty = k_full + L::kKSlots;
    uint64_t *v_full = k_empty + L::kKSlots, *v_empty = v_full + L::kVSlots;
    uint64_t *s_full = v_empty + L::kVSlots;  // per score buffer, as the next
    uint64_t *p_full = s_full + L::kBufs;
    uint64_t *o_final = p_full + L::kBufs;  // [2]: per softmax group
    uint64_t *pair_full = o_final + 2, *pair_read = pair_full + 1;
    uint64_t *unit_full = pair_read + 1, *unit_empty = unit_full + L::kUnits;
    uint64_t *drain = unit_empty + L::kUnits;
    volatile int *unit_slot = reinterpret_cast<volatile int *>(smem + L::kUnitOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMiscOff + 4);
    float2 *pair_ml = reinterpret_cast<float2 *>(smem + L::kPairOff);
    const int warp = warp_id(), lane = lane_id();
    const PagedWork work = {p.tile_toks, QT * p.tile_toks, paged_unit_cost(QT), p.causal};

    if (threadIdx.x == 96) {
        for (int s = 0; s < L::kKSlots; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < L::kVSlots; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&o_final[i], 1);
        }
        for (int i = 0; i < L::kBufs; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);  // one arrival per softmax warp of a group
        }
        for (int i = 0; i < L::kUnits; ++i) {
            mbar_init(&unit_full[i], 1);
            mbar_init(&unit_empty[i], 9);  // the MMA warp and the softmax warps
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
    // the plan is made by both load warps at once, so that V's does not wait for the other's slot
    PagedLine line;
    PagedCursor cur;
    long room = 0;
    PagedPiece own;  // CL: this CTA's share of its cluster's unit
    own.toks = 0;
    if (warp == 0 || warp == 2) {
        if constexpr (CL) {
            const int ctas = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
            if (find_unit(p.c, work, static_cast<int>(blockIdx.x) / ctas, blockIdx.x == 0 && warp == 0,
                          own)) {
                const int end = own.last0 + (p.causal ? own.toks - 1 : 0) + 1;  // keys it sees
                const int tiles = end > 0 ? (end + kPagedKeys - 1) / kPagedKeys : 0;
                own.t0 = rank * tiles / ctas;
                own.t1 = (rank + 1) * tiles / ctas;
            }
        } else {
            room = find_stretch(p.c, work, blockIdx.x == 0 && warp == 0, line, cur);
        }
    }
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
    // both groups work on the same query tile and take alternate key tiles
    auto is_pair = [&](int toks) { return QT == 1 || toks <= p.tile_toks; };
    // Q buffer of the nq-th piece with keys, and that buffer's tenants before it
    auto q_buf = [&](int nq) { return QT == 1 && p.q_bufs == 2 ? nq & 1 : 0; };
    auto q_use = [&](int nq) { return QT == 1 && p.q_bufs == 2 ? nq >> 1 : nq; };

    if (warp < 4) {
        // warpgroup 0 gives registers to the softmax groups: 128 x 88 + 256 x 208 = 64512, all of the
        // 384 x 168 = 64512 the CTA is launched with
        regs_dec<88>();
        const int box_rows = min(1 << p.c.page_shift, kPagedKeys);  // rows of one page in a tile
        const int boxes = kPagedKeys / box_rows;                    // pages of a tile
        if (warp == 0 || warp == 2) {
            // ------------------------------------------------- loads: Q and K, or V
            const bool is_v = warp == 2;
            const CUtensorMap *map = is_v ? &maps.v : &maps.k;
            uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
            uint8_t *ring = smem + (is_v ? L::kVOff : L::kKOff);
            const int slots = is_v ? L::kVSlots : L::kKSlots;
            int n = 0;  // tiles issued
            int slot = 0;
            uint32_t parity = 1;  // of the wait for the slot's last tenant
            int nq = 0;  // Q loads issued
            int k = 0;   // pieces so far
            bool ok = true;
            int4 cut0 = make_int4(-1, 0, 0, 0);  // what the merge has to do for this CTA
            int cut_n = 0;
            for (;;) {
                PagedPiece u;
                u.t0 = u.t1 = 0;
                long from = 0;
                bool any, whole;
                if constexpr (CL) {
                    u = own;
                    any = k == 0 && own.toks > 0;  // its share may be empty: it still joins the merge
                    whole = true;
                } else {
                    const long end = line.border(static_cast<int>(blockIdx.x) + 1);
                    while (room > 0) {
                        from = end - room;
                        u = cur.take(p.c, work, room);
                        if (u.t0 < u.t1) break;
                    }
                    any = u.t0 < u.t1;
                    whole = u.t1 - u.t0 == u.tiles;
                }
                const int first_tile = u.t0;
                // a unit that stands before its sequence sees nothing
                if (any && u.last0 + (p.causal ? u.toks - 1 : 0) < 0) u.t1 = u.t0;
                if (!is_v) {
                    const int e = k % L::kUnits;
                    if (k >= L::kUnits && !mbar_wait_warp(&unit_empty[e], (k / L::kUnits - 1) & 1,
                                                          p.ctl, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        volatile int *s = unit_slot + 8 * e;
                        s[0] = any ? u.tok0 : -1;
                        if (any) {
                            s[1] = u.toks;
                            s[2] = u.kvh;
                            s[3] = u.last0;
                            s[4] = u.len;
                            s[5] = u.t0;
                            s[6] = u.t1;
                            s[7] = CL ? kDestCluster
                                   : whole ? -1
                                         : 2 * static_cast<int>(blockIdx.x) + (first_tile == 0 ? 1 : 0);
                        }
                        mbar_arrive(&unit_full[e]);
                    }
                    __syncwarp();
                }
                if (!any) break;
                ++k;
                PageWindow win;
                win.open(p.c, u);
                auto load_q = [&]() {  // a Q buffer is free once its last unit's last S is done
                    const int buf = q_buf(nq), use = q_use(nq);
                    if (use > 0 && !mbar_wait_warp(&q_empty[buf], (use - 1) & 1, p.ctl, abort_flag))
                        return false;
                    if (lane == 0) {
                        const int tiles = is_pair(u.toks) ? 1 : 2;
                        mbar_arrive_expect_tx(
                            &q_full[buf], tiles * L::kBoxes * 128 * p.rep * p.q_box_toks);
                        for (int t = 0; t < tiles; ++t)
                            for (int b = 0; b < L::kBoxes; ++b)
                                tma_load_4d(smem + buf * kQBufBytes + t * L::kTileBytes +
                                                b * L::kBoxBytes,
                                            &maps.q, b * 64, 0, u.kvh, u.tok0 + t * p.tile_toks,
                                            &q_full[buf]);
                    }
                    ++nq;
                    return true;
                };
                bool q_done = is_v || u.t0 == u.t1;  // a piece that sees nothing needs no Q
                if (!q_done && nq == 0) ok = q_done = load_q();  // the first Q needs no page id
                for (int j = u.t0; j < u.t1 && ok; ++j) {
                    const int id = win.tile(p.c, j, boxes);
                    if (!mbar_wait_warp(&empty[slot], parity, p.ctl, abort_flag)) {
                        ok = false;
                        break;
                    }
                    // the tile's pages into its slot: one lane per page (test hook: not the first K)
                    const bool skip = p.ctl.fault_mode == 4 && !is_v && n == 0;
                    // K's rows behind the sequence's pages stay what they are: their scores are masked
                    const int used = is_v ? boxes : min(boxes, win.left(p.c, j));
                    if (lane == 0 && !skip)
                        mbar_arrive_expect_tx(&full[slot], used * box_rows * 128 * L::kBoxes);
                    __syncwarp();
                    if (lane < used && !skip) {
                        const int y = (j * kPagedKeys) & ((1 << p.c.page_shift) - 1);
                        uint8_t *dst = ring + slot * L::kTileBytes + lane * box_rows * 128;
                        for (int b = 0; b < L::kBoxes; ++b)
                            tma_load_4d(dst + b * L::kBoxBytes, map, b * 64,
                                        maps.rows_inner ? y : u.kvh, maps.rows_inner ? u.kvh : y,
                                        id, &full[slot]);
                    }
                    ++n;
                    if (++slot == slots) {
                        slot = 0;
                        parity ^= 1;
                    }
                    // the first K goes ahead of Q: its slot frees before the Q tiles do
                    if (!q_done) {
                        ok = load_q();
                        q_done = true;
                    }
                }
                if (!ok) break;
                if (!CL && !is_v && !whole && first_tile == 0) {  // a unit that other CTAs finish
                    cut0 = make_int4(u.tok0, u.toks, u.kvh, 0);
                    cut_n = line.holder(from + u.left - 1) - static_cast<int>(blockIdx.x) + 1;
                }
            }
            if (!CL && !is_v && p.cut != nullptr && lane == 0) {
                p.cut[2 * blockIdx.x] = cut0;
                p.cut[2 * blockIdx.x + 1] = make_int4(cut_n, 0, 0, 0);
            }
            if (!ok || *abort_flag) {
                // let every copy still in flight land before shared memory goes away
                if (lane == 0) {
                    for (int l = max(nq - (QT == 1 ? p.q_bufs : 1), 0); l < nq; ++l)
                        drain_wait(&q_full[q_buf(l)], q_use(l) & 1, p.ctl);
                    for (int l = n > slots ? n - slots : 0; l < n; ++l) {
                        if (p.ctl.fault_mode == 4 && !is_v && l == 0) continue;
                        drain_wait(&full[l % slots], (l / slots) & 1, p.ctl);
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------- MMA issuer
            const SDesc dq0 = sdesc_make(smem_u32(smem), 16, 1024);              // Q: K-major
            const SDesc dk0 = sdesc_make(smem_u32(smem + L::kKOff), 16, 1024);   // K: K-major
            const SDesc dv0 = sdesc_make(smem_u32(smem + L::kVOff), L::kBoxBytes,
                                         1024);                                   // V: MN-major
            auto issue_s = [&](int q, int buf, int ks) {  // q: where Q starts
                const SDesc a = sdesc_add(dq0, q);
                const SDesc b = sdesc_add(dk0, ks * L::kTileBytes);
                if constexpr (D == 128)
                    mma_ss_chain_k128(tmem + buf * 128, a, b, kIdescS, 0u);
                else
                    mma_ss_chain_k64(tmem + buf * 128, a, b, kIdescS, 0u);
                umma_commit_el(&s_full[buf]);
            };
            auto issue_pv = [&](int t, int buf, int vs, bool accumulate) {
                mma_ts_chain_k128(tmem + L::kOCol + t * D, tmem + buf * 128,
                                  sdesc_add(dv0, vs * L::kTileBytes), kIdescPV,
                                  accumulate ? 1u : 0u);
            };
            auto wait_ks = [&](int ks, uint32_t parity) {
                if (!mbar_wait_warp(&k_full[ks], parity, p.ctl, abort_flag)) return false;
                tc_fence_after();
                return true;
            };
            auto wait_k = [&](int x) { return wait_ks(x % L::kKSlots, (x / L::kKSlots) & 1); };
            // V tile x of the ring (key tile j) has landed; its rows from the sequence's end to
            // the end of that page become zeros (pages behind it were loaded as zeros)
            auto wait_vs = [&](int vs, uint32_t parity, int j, int len) {
                if (!mbar_wait_warp(&v_full[vs], parity, p.ctl, abort_flag)) return false;
                const int r0 = len - j * kPagedKeys;
                if (r0 < kPagedKeys) {
                    const int size = 1 << p.c.page_shift;
                    const int r1 = min(kPagedKeys, (r0 + size - 1) & ~(size - 1));
                    uint8_t *tile = smem + L::kVOff + vs * L::kTileBytes;
#pragma unroll 1
                    for (int b = 0; b < L::kBoxes; ++b)
#pragma unroll 1
                        for (int a = r0 * 128 + lane * 16; a < r1 * 128; a += 512)
                            *reinterpret_cast<uint4 *>(tile + b * L::kBoxBytes + a) =
                                make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                return true;
            };
            auto wait_v = [&](int x, int j, int len) {
                return wait_vs(x % L::kVSlots, (x / L::kVSlots) & 1, j, len);
            };
            int nq = 0;            // Q tiles used: pieces with keys
            int nt = 0;            // K and V tiles consumed
            int pcnt[2] = {0, 0};  // PV products per group (p_full phases)
            auto wait_p = [&](int t) {
                if (!mbar_wait_warp(&p_full[t], pcnt[t] & 1, p.ctl, abort_flag)) return false;
                tc_fence_after();
                return true;
            };
            // QT == 1: the key tiles of all pieces are one sequence, tile x for group x & 1 and score
            // buffer x mod kBufs, and PV of tile x - kBufs is issued before S of tile x, whichever
            // piece they belong to: the next piece's scores are under way while the last one's
            // probabilities are.
            struct Tile {
                int j, len;      // key tile (-1: none), the sequence's end
                bool add, last;  // not the first, the last of its group in the piece
            };
            Tile open[L::kBufs];  // tiles x - kBufs .. x - 1
#pragma unroll
            for (int i = 0; i < L::kBufs; ++i) open[i].j = -1;
            int nf = 0;                   // tiles finished: the number of open[0]
            int ks = 0, vs = 0;           // ring slots of tile x and of open[0]
            uint32_t kpar = 0, vpar = 0;  // parities of their barriers
            auto finish = [&]() {  // PV of open[0]
                if (open[0].j >= 0) {
                    const int g = nf & 1, buf = nf % L::kBufs;
                    if (!wait_vs(vs, vpar, open[0].j, open[0].len)) return false;
                    if (!mbar_wait_warp(&p_full[buf], (nf / L::kBufs) & 1, p.ctl, abort_flag))
                        return false;
                    tc_fence_after();
                    issue_pv(g, buf, vs, open[0].add);
                    if (open[0].last) umma_commit_el(&o_final[g]);
                    umma_commit_el(&v_empty[vs]);
                    if (++vs == L::kVSlots) {
                        vs = 0;
                        vpar ^= 1;
                    }
                    ++nf;
                }
#pragma unroll
                for (int i = 1; i < L::kBufs; ++i) open[i - 1] = open[i];
                open[L::kBufs - 1].j = -1;
                return true;
            };
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int e = k % L::kUnits;
                if (!mbar_wait_warp(&unit_full[e], (k / L::kUnits) & 1, p.ctl, abort_flag)) {
                    ok = false;
                    break;
                }
                const PieceSlot u = read_slot(e);
                if constexpr (QT == 1) {
                    const int buf = q_buf(nq);
                    // at the end, and at a piece that sees nothing, the open tiles are finished (the
                    // slot after next is free only then)
                    const int tiles = u.tok0 < 0 ? 0 : u.t1 - u.t0;
                    const int steps = tiles > 0 ? tiles : L::kBufs;
#pragma unroll 1
                    for (int i = 0; i < steps; ++i) {
                        if (!finish()) {
                            ok = false;
                            break;
                        }
                        if (tiles == 0) continue;
                        if ((i == 0 &&
                             !mbar_wait_warp(&q_full[buf], q_use(nq) & 1, p.ctl, abort_flag)) ||
                            !wait_ks(ks, kpar)) {
                            ok = false;
                            break;
                        }
                        issue_s(buf * kQBufBytes, nt % L::kBufs, ks);
                        umma_commit_el(&k_empty[ks]);
                        if (++ks == L::kKSlots) {
                            ks = 0;
                            kpar ^= 1;
                        }
                        if (i == tiles - 1) umma_commit_el(&q_empty[buf]);
                        open[L::kBufs - 1] = {u.t0 + i, u.len, i >= 2, i + 2 >= tiles};
                        ++nt;
                    }
                    if (!ok || u.tok0 < 0) break;
                    if (tiles > 0) ++nq;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&unit_empty[e]);
                    continue;
                }
                if (u.tok0 < 0) break;
                if (u.t0 < u.t1) {
                    if (!mbar_wait_warp(q_full, nq & 1, p.ctl, abort_flag)) {
                        ok = false;
                        break;
                    }
                    ++nq;
                    tc_fence_after();
                }
                const int p0[2] = {pcnt[0], pcnt[1]};
                const int n0 = nt - u.t0;  // ring index of key tile j is n0 + j
                if (is_pair(u.toks)) {
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
                                issue_pv(t, t, (n0 + jp) % L::kVSlots, pcnt[t] > p0[t]);
                                ++pcnt[t];
                                if (jp + 2 >= u.t1) umma_commit_el(&o_final[t]);
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
                                issue_pv(t, t, vs, pcnt[t] > p0[t]);
                                ++pcnt[t];
                                if (j == end[t]) umma_commit_el(&o_final[t]);
                            }
                            if (j < end[t]) issue_s(t * L::kTileBytes, t, (n0 + j) % L::kKSlots);
                        }
                        if (!ok) break;
                        if (j == u.t1 - 1) umma_commit_el(q_empty);
                        if (j > u.t0) umma_commit_el(&v_empty[vs]);
                        if (j < u.t1) umma_commit_el(&k_empty[(n0 + j) % L::kKSlots]);
                    }
                }
                if (!ok) break;
                nt += u.t1 - u.t0;
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
        const uint32_t tO = tmem + lane_base + L::kOCol + t * D;
        const float sl2 = p.scale_log2;
        int scnt = 0;          // score tiles consumed by this group
        int nfin = 0;          // pieces in which this group had products (o_final phases)
        int nfin1 = 0;         // the same of the other group
        int npair = 0;         // merges between the groups (pair_full, pair_read phases)
        bool owed = false;     // the other group has still to read what this one left in O_t
        int lead = 0;          // the group that has a pair's first key tile, and merges
        for (int k = 0;; ++k) {
            const int e = k % L::kUnits;
            if (!mbar_wait_warp(&unit_full[e], (k / L::kUnits) & 1, p.ctl, abort_flag)) break;
            const PieceSlot u = read_slot(e);
            if (u.tok0 < 0) break;
            const bool pair = is_pair(u.toks);
            const int q = pair ? 0 : t;  // query tile
            const bool leads = t == lead;
            // QT == 1: key tiles alternate between the groups across pieces too
            if (QT == 1) lead ^= (u.t1 - u.t0) & 1;
            const int first = u.t0 + (pair && !leads ? 1 : 0), step = pair ? 2 : 1;
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
                const int x = 2 * scnt + t, buf = L::kBufs == 2 ? t : x % L::kBufs;
                const uint32_t tS = tmem + lane_base + buf * 128;
                if (!mbar_wait_warp(&s_full[buf], (x / L::kBufs) & 1, p.ctl, abort_flag)) {
                    ok = false;
                    break;
                }
                ++scnt;
                tc_fence_after();
                // PV of this group's last tile, into O_t, is complete when its V slot is empty again
                auto o_ready = [&]() {
                    const int y = x - 2;
                    const bool in_time = mbar_wait_warp(&v_empty[y % L::kVSlots],
                                                        (y / L::kVSlots) & 1, p.ctl, abort_flag);
                    tc_fence_after();
                    return in_time;
                };
                if (QT == 1 && !CL && busy && u.t1 - u.t0 <= kShortPiece) {
                    // as below, in steps of 32 keys
                    const int lim = last - j * kPagedKeys;  // columns above lim are masked
                    float top = -INFINITY;
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        uint32_t r[32];
                        tmem_ld32(tS + 32 * h, r);
                        tmem_wait_ld();
                        const int limh = lim - 32 * h;
                        if (limh < 31) {
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (c > limh) r[c] = __float_as_uint(-INFINITY);
                        }
                        float mx[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            mx[c] = fmaxf(fmax3(__uint_as_float(r[c]), __uint_as_float(r[4 + c]),
                                                __uint_as_float(r[8 + c])),
                                          fmax3(fmaxf(__uint_as_float(r[12 + c]),
                                                      __uint_as_float(r[16 + c])),
                                                fmaxf(__uint_as_float(r[20 + c]),
                                                      __uint_as_float(r[24 + c])),
                                                __uint_as_float(r[28 + c])));
                        top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                    }
                    const float m_new = fmaxf(m, top * sl2);
                    bool rescale = false;
                    float alpha = 1.f;
                    if (m_new > m + 8.0f) {
                        rescale = m != -INFINITY;
                        if (rescale) alpha = ex2(m - m_new);
                        l *= alpha;
                        m = m_new;
                    }
                    const float mu = m == -INFINITY ? 0.f : m;  // nothing unmasked yet
                    float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                     make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    const float2 sc2 = make_float2(sl2, sl2), mu2 = make_float2(-mu, -mu);
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        uint32_t r[32], pk[16];
                        tmem_ld32(tS + 32 * h, r);
                        tmem_wait_ld();
                        const int limh = lim - 32 * h;
                        if (limh < 31) {
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (c > limh) r[c] = __float_as_uint(-INFINITY);
                        }
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float2 x = ffma2(make_float2(__uint_as_float(r[2 * c]),
                                                               __uint_as_float(r[2 * c + 1])),
                                                   sc2, mu2);
                            const float2 ev = make_float2(ex2(x.x), ex2(x.y));
                            acc[c & 3] = fadd2(acc[c & 3], ev);
                            pk[c] = pack2<BF16>(ev.x, ev.y);
                        }
                        tmem_st16(tS + 16 * h, pk);  // over scores that are done with
                    }
                    const float2 a = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
                    l += a.x + a.y;
                    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
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
                } else if (busy) {
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
                        // the previous PV into O_t is complete (with two score buffers it was before
                        // this S_t), and the next one waits for p_full, so O_t is ours to rescale
                        if (L::kBufs == 3 && !o_ready()) {
                            ok = false;
                            break;
                        }
#pragma unroll 1
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
                if (owed) {  // this arrival lets the next PV overwrite what was left in O_t
                    if (!mbar_wait_warp(pair_read, (npair - 1) & 1, p.ctl, abort_flag)) {
                        ok = false;
                        break;
                    }
                    owed = false;
                }
                mbar_arrive_warp_after_st(&p_full[buf]);
            }
            if (!ok) break;
            const bool had = first < end;
            const bool both = pair && u.t1 - u.t0 > 1;  // the second group has a share
            if (pair && !leads) {
                if (both) {  // its statistics for the leading group, which finds O_t in place
                    pair_ml[row] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pair_full);
                    ++npair;
                    ++nfin;
                    owed = true;
                }
                if (u.t0 < u.t1) ++nfin1;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&unit_empty[e]);
                continue;
            }
            if (had) {
                if (!mbar_wait_warp(&o_final[t], nfin & 1, p.ctl, abort_flag)) break;
                ++nfin;
            }
            if constexpr (CL && QT == 2) {
                // the results go over the K and V rings: the other group's products are done too (a
                // CTA has one piece, so this is that barrier's first phase)
                if (!pair && piece_end(u, 1 - t, p.tile_toks, p.causal) > u.t0 &&
                    !mbar_wait_warp(&o_final[1 - t], 0, p.ctl, abort_flag))
                    break;
            }
            float wa = 1.f, wb = 0.f;  // weights of this group's O and of the other's
            if (both) {
                if (!mbar_wait_warp(pair_full, npair & 1, p.ctl, abort_flag)) break;
                if (!mbar_wait_warp(&o_final[1 - t], nfin1 & 1, p.ctl, abort_flag)) break;
                ++npair;
                ++nfin1;
                const float2 o = pair_ml[row];
                const float M = fmaxf(m, o.x), mu = M == -INFINITY ? 0.f : M;
                wa = ex2(m - mu);
                wb = ex2(o.x - mu);
                l = l * wa + o.y * wb;
                m = M;
            } else if (!pair && piece_end(u, 1 - t, p.tile_toks, p.causal) > u.t0) {
                ++nfin1;  // the other group waits for its own
            }
            tc_fence_after();
            if (busy) {
                // O and LSE, or the piece's partial (m, l, O~); the tensor-memory loads are
                // warp-wide, the stores only for real rows
                const float inv = CL || u.dest >= 0 ? 1.f : l > 0.f ? 1.f / l : 0.f;
                wa *= inv;
                wb *= inv;
                const int head = u.kvh * p.rep + row_head;
                const long otok = u.tok0 + tok;
                const int prow = q * 128 + row;
                // (rolled up, as what else runs once a unit: unrolled, a mixed batch takes 50.7 us and
                // not 48.8, 1024 sequences of up to 500 keys 314 and not 306)
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32], o1[32];
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
                        tmem_ld32(tO + (t == 0 ? D : -D) + cc * 32, o1);  // the other's
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            o[x] = __float_as_uint(
                                fmaf(__uint_as_float(o1[x]), wb, __uint_as_float(o[x])));
                    }
                    if (!real) continue;
                    if constexpr (CL) {
                        float4 *dst = reinterpret_cast<float4 *>(
                            smem + L::kKOff + (q * 128 + row) * L::kRowBytes + cc * 128);
#pragma unroll
                        for (int q4 = 0; q4 < 8; ++q4)
                            dst[q4] = make_float4(
                                __uint_as_float(o[4 * q4]), __uint_as_float(o[4 * q4 + 1]),
                                __uint_as_float(o[4 * q4 + 2]), __uint_as_float(o[4 * q4 + 3]));
                    } else if (u.dest < 0) {
                        uint4 *dst = reinterpret_cast<uint4 *>(
                            reinterpret_cast<T *>(p.o) + otok * p.o_t + head * p.o_h + cc * 32);
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4) {
                            // a row that sees no key is zero, though a zero probability met the
                            // values that the unit's other rows see and one of them is not finite
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                w[x] = l == 0.f ? 0u
                                                : pack2<BF16>(__uint_as_float(o[8 * q4 + 2 * x]),
                                                              __uint_as_float(o[8 * q4 + 2 * x + 1]));
                            dst[q4] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        // column-major in groups of four: the warp's rows side by side, 512 bytes
                        // a store (row by row the 256 rows took 11000 cycles)
                        float4 *dst = p.part_o +
                                      (static_cast<long>(u.dest) * (D / 4) + cc * 8) * p.part_rows + prow;
#pragma unroll
                        for (int q4 = 0; q4 < 8; ++q4)
                            dst[q4 * p.part_rows] = make_float4(
                                __uint_as_float(o[4 * q4]), __uint_as_float(o[4 * q4 + 1]),
                                __uint_as_float(o[4 * q4 + 2]), __uint_as_float(o[4 * q4 + 3]));
                    }
                }
                if (CL) {  // over the Q tiles
                    reinterpret_cast<float2 *>(smem)[q * 128 + row] = make_float2(m, l);
                } else if (real) {
                    if (u.dest < 0)
                        p.lse[otok * p.c.H + head] = row_lse(m, l);
                    else
                        p.part_ml[static_cast<long>(u.dest) * p.part_rows + prow] = make_float2(m, l);
                }
            }
            // O has been read out (the next unit's first PV into it waits for this warp's next
            // p_full arrival, or the other group's after pair_read)
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
    if constexpr (CL) {
        // the cluster's CTAs hold (m, l, O~) of their shares; each of them merges a slice of the
        // rows' columns, in rank order
        const unsigned ctas = cluster_size();
        cluster_sync();
        const PieceSlot u = read_slot(0);
        const int items = u.tok0 < 0 ? 0 : u.toks * p.rep * (D / 4);
        const uint32_t ml0 = smem_u32(smem), o0 = smem_u32(smem + L::kKOff);
        for (int i = static_cast<int>(cluster_rank() * L::kThreads + threadIdx.x); i < items;
             i += static_cast<int>(ctas * L::kThreads)) {
            const int col = i % (D / 4), which = i / (D / 4);  // 4 columns of one token's head
            const int tok = which / p.rep, h = which - tok * p.rep;
            const int q = QT == 2 && tok >= p.tile_toks ? 1 : 0;
            const int row = q * 128 + (tok - q * p.tile_toks) * p.rep + h;
            float2 ml[kMaxCluster];
            float4 x[kMaxCluster];
            float M = -INFINITY;
#pragma unroll
            for (unsigned r = 0; r < kMaxCluster; ++r) {
                ml[r] = make_float2(-INFINITY, 0.f);
                if (r < ctas) {
                    ml[r] = cluster_ld2(cluster_map(ml0 + row * 8, r));
                    x[r] = cluster_ld4(cluster_map(o0 + row * L::kRowBytes + col * 16, r));
                }
                M = fmaxf(M, ml[r].x);
            }
            const float mu = M == -INFINITY ? 0.f : M;
            float l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (unsigned r = 0; r < kMaxCluster; ++r) {
                // a share that saw nothing weighs nothing, one that is all NaN passes it on
                if (r >= ctas || ml[r].y == 0.f) continue;
                const float w = ml[r].x == -INFINITY ? 1.f : ex2(ml[r].x - mu);
                l = fmaf(w, ml[r].y, l);
                acc = make_float4(fmaf(w, x[r].x, acc.x), fmaf(w, x[r].y, acc.y),
                                  fmaf(w, x[r].z, acc.z), fmaf(w, x[r].w, acc.w));
            }
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const long otok = u.tok0 + tok;
            const int head = u.kvh * p.rep + h;
            *reinterpret_cast<uint2 *>(p.o + otok * p.o_t + head * p.o_h + col * 4) = make_uint2(
                pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
            if (col == 0) p.lse[otok * p.c.H + head] = row_lse(M, l);
        }
        cluster_sync();  // no CTA leaves while another still reads its shared memory
    }
}

// Merge of the units that borders cut: block (c, y) does rows [32 y, 32 y + 32) of the unit whose first
// piece CTA c ended with, a lane per row and a slice of the columns per warp.  The pieces stand in
// CTA order and are folded in in that order (deterministic), a batch at a time with all its reads
// in flight: M = max m_s, w_s = 2^(m_s - M), l = sum w_s l_s, O = sum w_s O_s / l, LSE = (M + log2 l) ln 2.
// A chunk's unit has 256 rows in few pieces, so its batches are small and more blocks share an SM; a
// single token's unit has few rows in up to one piece per SM.
constexpr int kMergeWarps = 8;
template <int D, bool BF16, int QT>
__global__ void __launch_bounds__(kMergeWarps * 32) fa_paged_merge_kernel(const PagedAttnParams p) {
    using T = elem_t<BF16>;
    constexpr int kCols = D / 4 / kMergeWarps;  // float4 columns per warp
    constexpr int kBatch = QT == 2 ? 2 : 8;
    griddep_wait();
    const int c = static_cast<int>(blockIdx.x), warp = warp_id();
    const int4 cut = p.cut[2 * c];
    const int pieces = p.cut[2 * c + 1].x;
    if (pieces < 2) return;
    const int tok0 = cut.x, toks = cut.y, kvh = cut.z;
    const int r = static_cast<int>(blockIdx.y) * 32 + lane_id();
    const int row = r & 127, row_tok = row / p.rep, tok = (r >> 7) * p.tile_toks + row_tok;
    if (r >= p.part_rows || row_tok >= p.tile_toks || tok >= toks) return;
    float M = -INFINITY, l = 0.f;
    float4 acc[kCols];
#pragma unroll
    for (int e = 0; e < kCols; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < pieces; s0 += kBatch) {
        float2 ml[kBatch];
        float4 x[kBatch][kCols];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            ml[i] = make_float2(-INFINITY, 0.f);
            if (s0 + i < pieces) {
                const long slot = s0 + i == 0 ? 2 * c + 1 : 2 * (c + s0 + i);
                ml[i] = p.part_ml[slot * p.part_rows + r];
                const float4 *src = p.part_o + (slot * (D / 4) + warp * kCols) * p.part_rows + r;
#pragma unroll
                for (int e = 0; e < kCols; ++e) x[i][e] = src[e * p.part_rows];
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
        for (int e = 0; e < kCols; ++e)
            acc[e] = make_float4(acc[e].x * back, acc[e].y * back, acc[e].z * back, acc[e].w * back);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            // a piece that saw nothing (l = 0) weighs nothing; one whose scores are all NaN
            // (m = -inf, l = NaN) passes its NaN on
            if (s0 + i >= pieces || ml[i].y == 0.f) continue;
            const float w = ml[i].x == -INFINITY ? 1.f : ex2(ml[i].x - mu);
            l = fmaf(w, ml[i].y, l);
#pragma unroll
            for (int e = 0; e < kCols; ++e)
                acc[e] = make_float4(fmaf(w, x[i][e].x, acc[e].x), fmaf(w, x[i][e].y, acc[e].y),
                                     fmaf(w, x[i][e].z, acc[e].z), fmaf(w, x[i][e].w, acc[e].w));
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int head = kvh * p.rep + row % p.rep;
    uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<T *>(p.o) +
                                           static_cast<long>(tok0 + tok) * p.o_t + head * p.o_h +
                                           warp * kCols * 4);
#pragma unroll
    for (int e = 0; e < kCols; e += 2)
        dst[e / 2] = make_uint4(pack2<BF16>(acc[e].x * inv, acc[e].y * inv),
                                pack2<BF16>(acc[e].z * inv, acc[e].w * inv),
                                pack2<BF16>(acc[e + 1].x * inv, acc[e + 1].y * inv),
                                pack2<BF16>(acc[e + 1].z * inv, acc[e + 1].w * inv));
    if (warp == 0) p.lse[static_cast<long>(tok0 + tok) * p.c.H + head] = row_lse(M, l);
}

// The dynamic shared memory of a kernel, allowed once per device (the attribute holds from then on).
cudaError_t allow_smem(std::atomic<unsigned long long> &ready, const void *kernel, int bytes,
                       int device) {
    const unsigned long long bit = 1ull << (device & 63);
    if ((ready.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
    return e;
}

template <int D, bool BF16, int QT>
cudaError_t launch_line(const PagedMaps &m, const PagedAttnParams &p, cudaStream_t stream) {
    using L = PagedLayout<D, QT, false>;
    auto kern = fa_paged_attn_kernel<D, BF16, QT, false>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = allow_smem(ready, reinterpret_cast<const void *>(kern), L::kAlloc, p.device);
    if (e != cudaSuccess) return e;
    // not launched to overlap the grid before it: its CTAs would then take the SMs in the order in
    // which they come free, prompt chunks and single tokens no longer spread over the chip (when tried, a
    // mixed batch 51.8 -> 56.6 us, a single sequence 11.0 -> 10.2)
    kern<<<kPagedCtas, L::kThreads, L::kAlloc, stream>>>(m, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.cut == nullptr) return e;
    // (the host does not know whether a unit was cut: where none was, this grid costs 0.6 us)
    return launch_overlapped(fa_paged_merge_kernel<D, BF16, QT>,
                             dim3(kPagedCtas - 1, (p.part_rows + 31) / 32), kMergeWarps * 32, 0,
                             stream, p);
}

template <int D, bool BF16, int QT>
cudaError_t launch_clusters(const PagedMaps &m, const PagedAttnParams &p, PagedClusters cl,
                            cudaStream_t stream) {
    using L = PagedLayout<D, QT, true>;
    auto kern = fa_paged_attn_kernel<D, BF16, QT, true>;
    static std::atomic<unsigned long long> ready{0};
    const cudaError_t e = allow_smem(ready, reinterpret_cast<const void *>(kern), L::kAlloc, p.device);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cl.units * cl.ctas));
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = L::kAlloc;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cl.ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, m, p);
}

template <int D, bool BF16>
cudaError_t launch_attn_t(const PagedMaps &m, const PagedAttnParams &p, int tiles, PagedClusters cl,
                          cudaStream_t st) {
    if (cl.ctas > 0) return tiles == 2 ? launch_clusters<D, BF16, 2>(m, p, cl, st)
                                       : launch_clusters<D, BF16, 1>(m, p, cl, st);
    return tiles == 2 ? launch_line<D, BF16, 2>(m, p, st) : launch_line<D, BF16, 1>(m, p, st);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedMaps &m, const PagedAttnParams &p, int d, bool bf16,
                              int tiles, PagedClusters cl, cudaStream_t stream) {
    if (d == 64) return bf16 ? launch_attn_t<64, true>(m, p, tiles, cl, stream)
                             : launch_attn_t<64, false>(m, p, tiles, cl, stream);
    return bf16 ? launch_attn_t<128, true>(m, p, tiles, cl, stream)
                : launch_attn_t<128, false>(m, p, tiles, cl, stream);
}

}  // namespace fa
