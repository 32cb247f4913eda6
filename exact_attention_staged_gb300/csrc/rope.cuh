// rope.cuh - the rotation of rotary positions, shared by the rope and the paged-append kernels.
//
// Pair j of a row at position p is turned by the angle p * f_j.  f_j comes as turns per position
// in units of 2^-64 turns, so p * f_j modulo one turn is the low 64 bits of an integer product:
// no rounding at any position (a 32-bit float angle is off by 0.06 rad at position 10^6), and no
// 64-bit floating point, whose rate on this GPU is 1/64 of the 32-bit one.  The top 32 bits of the
// product are the angle, cut to 2^-32 turns (2^-29.4 radians) and rounded to 24 bits (below 2^-22.3
// radians up to pi, 2^-23 of a small angle).  Its sine and cosine come from the special-function unit,
// whose errors in [-pi, pi) are absolute: 2^-21.4 and 2^-21.2, which with the angle's are below 2^-20.6
// of a pair's size, 1/3100 and 1/390 of the rounding to bf16 and fp16 that follows.  Most pairs of
// a row turn by little over a whole prompt, and where such a sine stands alone (its pair's other
// element is zero or small) an absolute error would be up to 12 half units of the result, so below
// 1/4 it is the Taylor series to t^5, 2^-24 relative.  The accurate functions took about 25
// instructions a pair, which bounded rows of few heads; the series takes six (378 tokens appended
// 3.55 -> 3.7 us, rope the same).
#pragma once

#include "positions.h"

namespace fa {

constexpr int kRopePairs = 8;   // pairs per thread: two 16-byte pieces of a row
constexpr int kRopeElems = 16;

// cos and sin (times mscale) of the 8 pairs that start at pair `first`.
__device__ __forceinline__ void rope_angles(const unsigned long long *freq, int first, int pos,
                                            float mscale, float *cs, float *sn) {
    const ulonglong2 *src = reinterpret_cast<const ulonglong2 *>(freq + first);
    const unsigned long long p = static_cast<unsigned long long>(static_cast<long long>(pos));
#pragma unroll
    for (int j = 0; j < kRopePairs / 2; ++j) {
        const ulonglong2 f = src[j];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const unsigned long long turns = (e ? f.y : f.x) * p;
            // signed, so that the angle lies in [-pi, pi) and small ones keep their bits
            const int top = static_cast<int>(turns >> 32);
            const float angle = static_cast<float>(top) * 1.4629180792671596e-9f;  // 2 pi / 2^32
            const float x2 = angle * angle;
            const float series = angle * fmaf(x2, fmaf(x2, 1.f / 120.f, -1.f / 6.f), 1.f);
            cs[2 * j + e] = __cosf(angle) * mscale;
            sn[2 * j + e] = (fabsf(angle) < 0.25f ? series : __sinf(angle)) * mscale;
        }
    }
}

// The 8 pairs of one thread: (a, b) -> (a cos - b sin, b cos + a sin), in fp32, rounded once.
// lo, hi: the first and the second 16 bytes; with interleaved pairs a pair is two neighbouring
// elements, otherwise element i of lo goes with element i of hi.
template <bool BF16, bool INTER>
__device__ __forceinline__ void rope_turn(uint4 &lo, uint4 &hi, const float *cs, const float *sn) {
    uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if constexpr (INTER) {  // word w of lo is pair w, of hi pair 4 + w
            const float2 x = unpack2<BF16>(a[w]), y = unpack2<BF16>(b[w]);
            a[w] = pack2<BF16>(x.x * cs[w] - x.y * sn[w], x.y * cs[w] + x.x * sn[w]);
            b[w] = pack2<BF16>(y.x * cs[4 + w] - y.y * sn[4 + w], y.y * cs[4 + w] + y.x * sn[4 + w]);
        } else {  // words w of lo and hi hold pairs 2w and 2w + 1
            const float2 x = unpack2<BF16>(a[w]), y = unpack2<BF16>(b[w]);
            a[w] = pack2<BF16>(x.x * cs[2 * w] - y.x * sn[2 * w],
                               x.y * cs[2 * w + 1] - y.y * sn[2 * w + 1]);
            b[w] = pack2<BF16>(y.x * cs[2 * w] + x.x * sn[2 * w],
                               y.y * cs[2 * w + 1] + x.y * sn[2 * w + 1]);
        }
    }
    lo = make_uint4(a[0], a[1], a[2], a[3]);
    hi = make_uint4(b[0], b[1], b[2], b[3]);
}

// Elements where the two 16-byte pieces of unit u of a row start: units below rot / 16 hold 8
// pairs, the others are 16 elements that pass through.
template <bool INTER>
__device__ __forceinline__ int2 rope_pieces(int u, int rot) {
    if (INTER || u * kRopeElems >= rot) return make_int2(u * kRopeElems, u * kRopeElems + 8);
    return make_int2(u * kRopePairs, rot / 2 + u * kRopePairs);
}

}  // namespace fa
