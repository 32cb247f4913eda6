// fa_rope.cu - rotary positions on Q and K, forward and backward.
//
// Row n of head h of batch b at position p = positions[b][n]: every pair (a, c) of its first
// rot_dim elements becomes (a cos t - c sin t, c cos t + a sin t) times mscale, t = p f_j; the
// elements behind rot_dim are copied.  The backward is the transpose: the same with -t.
//
// The work is one read and one write of every element, 6 operations a pair, so it is bound by
// HBM: 8192 rows of 40 heads of 128 take 27.1 us, 6.2 TB/s or 0.91 of the measured copy rate.  A
// thread owns one unit of a row (8 pairs, or 16 elements that pass through) and walks
// the heads of a chunk: their angle is the same, so the sines and cosines are worked out once for
// all of them (Q's and K's heads alike: one launch for both), and the loads of several heads are
// in flight at a time.
#include "rope.cuh"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // heads whose loads are in flight together

template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 3) fa_rope_kernel(const RopeParams p) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kUnits = D / kRopeElems;  // units of a row
    const int u = static_cast<int>(threadIdx.x) % kUnits;
    const long row = static_cast<long>(blockIdx.x) * (kRopeThreads / kUnits) + threadIdx.x / kUnits;
    if (row >= p.rows) return;
    const int b = static_cast<int>(row / p.N), n = static_cast<int>(row - static_cast<long>(b) * p.N);
    const bool turn = u * kRopeElems < p.rot;
    float cs[kRopePairs], sn[kRopePairs];
    if (turn) {
        const int pos = p.positions != nullptr ? p.positions[row] : n;
        rope_angles(p.freq, u * kRopePairs, pos, p.mscale, cs, sn);
        if (p.inverse)
#pragma unroll
            for (int j = 0; j < kRopePairs; ++j) sn[j] = -sn[j];
    }
    const int2 at = rope_pieces<INTER>(u, p.rot);
    const int h0 = static_cast<int>(blockIdx.y) * p.chunk, h1 = min(h0 + p.chunk, p.H + p.Hkv);
    for (int h = h0; h < h1; h += kRopeBatch) {
        uint4 lo[kRopeBatch], hi[kRopeBatch];
        uint16_t *dst[kRopeBatch];
#pragma unroll
        for (int i = 0; i < kRopeBatch; ++i) {
            if (h + i >= h1) break;
            const bool isq = h + i < p.H;
            const int hh = isq ? h + i : h + i - p.H;
            const RopeSide &s = isq ? p.q : p.k;
            const uint16_t *src = s.in + b * s.in_b + hh * s.in_h + n * s.in_n;
            dst[i] = s.out + b * s.out_b + hh * s.out_h + n * s.out_n;
            lo[i] = __ldcs(reinterpret_cast<const uint4 *>(src + at.x));
            hi[i] = __ldcs(reinterpret_cast<const uint4 *>(src + at.y));
        }
#pragma unroll
        for (int i = 0; i < kRopeBatch; ++i) {
            if (h + i >= h1) break;
            if (turn) rope_turn<BF16, INTER>(lo[i], hi[i], cs, sn);
            *reinterpret_cast<uint4 *>(dst[i] + at.x) = lo[i];
            *reinterpret_cast<uint4 *>(dst[i] + at.y) = hi[i];
        }
    }
}

template <int D, bool BF16, bool INTER>
cudaError_t launch_rope_t(RopeParams p, cudaStream_t stream) {
    const long per_block = kRopeThreads / (D / kRopeElems);
    const long blocks = (p.rows + per_block - 1) / per_block;
    // heads per thread: two batches of them while that leaves every SM four blocks (one more than it
    // holds), else one, else fewer heads.  8k x 40 heads: 27.0 us against 30.4 with five heads and
    // twice the blocks; 1k x 32 heads of 64: 8.2 against 10.7 with one head and twice the blocks.  It does
    // not look at waves: 4092 rows of 32 heads of 64 are 1024 blocks, 2.25 times the 456 that fit.
    const int heads = p.H + p.Hkv;
    p.chunk = 2 * kRopeBatch;
    while (p.chunk > 1 && blocks * ((heads + p.chunk - 1) / p.chunk) < 4 * 152) p.chunk /= 2;
    dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + p.chunk - 1) / p.chunk));
    return launch_overlapped(fa_rope_kernel<D, BF16, INTER>, grid, kRopeThreads, 0, stream, p);
}

template <int D>
cudaError_t launch_rope_d(const RopeParams &p, bool bf16, bool inter, cudaStream_t stream) {
    if (bf16) return inter ? launch_rope_t<D, true, true>(p, stream)
                           : launch_rope_t<D, true, false>(p, stream);
    return inter ? launch_rope_t<D, false, true>(p, stream)
                 : launch_rope_t<D, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int d, bool bf16, bool inter, cudaStream_t stream) {
    return d == 64 ? launch_rope_d<64>(p, bf16, inter, stream)
                   : launch_rope_d<128>(p, bf16, inter, stream);
}

}  // namespace fa
