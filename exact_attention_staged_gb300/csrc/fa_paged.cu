// fa_paged.cu - the paged K/V cache: appending new tokens to it.
//
// A cache is a pool of pages, each with page_size rows of every K/V head; a sequence's table
// names its pages in order.  Token i of the n new tokens of sequence b stands at position
// p = kv_len[b] - n + i: its K, rotated to p, and its V go to row p mod page_size of page
// table[b][p div page_size], and its Q is rotated to p beside them.
//
// The work is one read and one write of every element of Q, K and V of the new tokens: bound by
// HBM for prompt chunks and by the latency of the index reads for a token or two.  A warp takes
// one token and a chunk of its heads; neighbouring lanes hold neighbouring pieces of a row, and
// the data is loaded before the token's sequence, length and page are looked up, so that the two
// chains of reads overlap.
#include "paged.cuh"
#include "rope.cuh"

namespace fa {
namespace {

constexpr int kAppendWarps = 8;
constexpr int kAppendBatch = 2;  // row pieces of a lane in flight together

template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kAppendWarps * 32, 4) fa_paged_append_kernel(const PagedAppendParams p) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kUnits = D / kRopeElems;   // units of a row
    constexpr int kHeads = 32 / kUnits;      // heads that a warp takes at a time
    const PagedView &c = p.c;
    if (blockIdx.x >= p.blocks) {  // every sequence's entries are looked at, also without a token
        const long b = static_cast<long>(blockIdx.x - p.blocks) * (kAppendWarps * 32) + threadIdx.x;
        if (b < c.B && paged_seq(c, static_cast<int>(b)).bad) paged_report(c);
        return;
    }
    const long w = static_cast<long>(blockIdx.x) * kAppendWarps + warp_id();
    const long token = w / p.chunks;
    if (token >= c.T) return;
    const int t = static_cast<int>(token);
    const int u = lane_id() % kUnits, hs = lane_id() / kUnits;
    const int heads_q = p.q != nullptr ? c.H : 0;
    const int heads = heads_q + 2 * c.Hkv;  // Q's, K's and V's
    const int rot = p.freq != nullptr ? p.rot : 0;
    const bool turn = u * kRopeElems < rot;
    const int2 at = rope_pieces<INTER>(u, rot);
    const int step = p.chunks * kHeads;
    const int first = static_cast<int>(w - token * p.chunks) * kHeads + hs;

    int b = -1, pos = -1, page = -1;
    bool known = false, skip = false;
    float cs[kRopePairs], sn[kRopePairs];
    // every lane runs the same number of rounds: the look-up below is warp-wide
    const int rounds = (heads + step - 1) / step;
    for (int r0 = 0; r0 < rounds; r0 += kAppendBatch) {
        uint4 lo[kAppendBatch], hi[kAppendBatch];
#pragma unroll
        for (int i = 0; i < kAppendBatch; ++i) {
            const int h = first + (r0 + i) * step;
            if (h >= heads) continue;
            const bool isq = h < heads_q, isk = h < heads_q + c.Hkv;
            const uint16_t *src = isq ? p.q + t * p.q_t + h * p.q_h
                                  : isk ? p.k + t * p.k_t + (h - heads_q) * p.k_h
                                        : p.v + t * p.v_t + (h - heads_q - c.Hkv) * p.v_h;
            const int2 from = h < heads_q + c.Hkv ? at : make_int2(u * kRopeElems, u * kRopeElems + 8);
            lo[i] = __ldcs(reinterpret_cast<const uint4 *>(src + from.x));
            hi[i] = __ldcs(reinterpret_cast<const uint4 *>(src + from.y));
        }
        if (!known) {
            known = true;
            b = paged_find(c, t);
            if (b < 0) return;  // no sequence's token: nothing of it is written
            const PagedSeq s = paged_seq(c, b);
            const int i = t - s.tok0;
            if (i < 0 || i >= s.n) return;
            pos = s.ctx + i;
            // before the sequence a token has no row in the cache; a length or offset out of range
            // was clamped, so the rows that it would name are not the sequence's
            skip = pos < 0 || s.bad;
            if (!skip) {
                page = paged_page(c, b, pos);
                if (page < 0) {
                    skip = true;
                    if (lane_id() == 0) paged_report(c);
                }
            }
            if (turn)
                rope_angles(p.freq, u * kRopePairs, p.positions != nullptr ? p.positions[t] : pos,
                            p.mscale, cs, sn);
        }
        const long row = pos & ((1 << c.page_shift) - 1);
#pragma unroll
        for (int i = 0; i < kAppendBatch; ++i) {
            const int h = first + (r0 + i) * step;
            if (h >= heads) continue;
            const bool isq = h < heads_q, isk = h < heads_q + c.Hkv;
            if (!isq && skip) continue;
            uint16_t *dst = isq ? p.q_out + t * p.qo_t + h * p.qo_h
                            : isk ? p.k_pages + page * p.kp_p + (h - heads_q) * p.kp_h + row * p.kp_r
                                  : p.v_pages + page * p.vp_p + (h - heads_q - c.Hkv) * p.vp_h +
                                        row * p.vp_r;
            const bool turned = h < heads_q + c.Hkv;  // V is stored as it is
            const int2 to = turned ? at : make_int2(u * kRopeElems, u * kRopeElems + 8);
            if (turned && turn) rope_turn<BF16, INTER>(lo[i], hi[i], cs, sn);
            *reinterpret_cast<uint4 *>(dst + to.x) = lo[i];
            *reinterpret_cast<uint4 *>(dst + to.y) = hi[i];
        }
    }
}

template <int D, bool BF16, bool INTER>
cudaError_t launch_append_t(PagedAppendParams p, cudaStream_t stream) {
    constexpr int kHeads = 32 / (D / kRopeElems);
    const int heads = (p.q != nullptr ? p.c.H : 0) + 2 * p.c.Hkv;
    const int rounds = (heads + kHeads - 1) / kHeads;
    // a token's heads are spread over several warps while there are few tokens
    int per = rounds;
    while (per > 1 && static_cast<long>(p.c.T) * ((rounds + per - 1) / per) < 152 * 64)
        per = (per + 1) / 2;
    p.chunks = (rounds + per - 1) / per;
    const long warps = static_cast<long>(p.c.T) * p.chunks;
    p.blocks = static_cast<unsigned>((warps + kAppendWarps - 1) / kAppendWarps);
    // blocks behind these look for bad entries, a thread per sequence (16 tokens take 3.05 us, 3.09
    // without them)
    const unsigned grid = p.blocks + (static_cast<unsigned>(p.c.B) - 1) / (kAppendWarps * 32) + 1;
    return launch_overlapped(fa_paged_append_kernel<D, BF16, INTER>, dim3(grid), kAppendWarps * 32, 0,
                             stream, p);
}

template <int D>
cudaError_t launch_append_d(const PagedAppendParams &p, bool bf16, bool inter, cudaStream_t st) {
    if (bf16) return inter ? launch_append_t<D, true, true>(p, st)
                           : launch_append_t<D, true, false>(p, st);
    return inter ? launch_append_t<D, false, true>(p, st) : launch_append_t<D, false, false>(p, st);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams &p, int d, bool bf16, bool inter,
                                cudaStream_t stream) {
    return d == 64 ? launch_append_d<64>(p, bf16, inter, stream)
                   : launch_append_d<128>(p, bf16, inter, stream);
}

}  // namespace fa
