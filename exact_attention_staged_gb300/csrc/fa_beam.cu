// fa_beam.cu - beam search's selection over beams and vocabulary.
//
// Candidate (w, v) of a request continues beam w with token v and scores
//   s(w, v) = score_w + x_wv - L_w,   L_w = ln sum_v e^x_wv,
// and the K best of the W V candidates are wanted, equal ones by the lowest w V + v.  Within a row the
// order of s is that of x, so a row's logits are read once: a CTA streams a piece of a row, tile after
// tile with the next one's loads in flight, and keeps the sum of e^(x - m) with a running maximum m per
// thread (fp32); a second, small grid joins the pieces' statistics and candidates of a request.  Where the
// logits are many times L2, reading them is most of it (1024 rows of 131072 fp32 97 us, 0.82 of the copy
// bandwidth; of bf16 55 us, 0.71).  256 rows of 131072 bf16 take 18 us, and the 14.4 of streaming as long where the loop
// forms nothing but maxima: what bounds it is neither arithmetic nor HBM (3.7 TB/s, from L2 in part) but what is
// in flight, 64 bytes of a thread, one tile ahead and 512 CTAs in 608 places, and the launch.
//
// The K largest of a piece: while streaming, a thread only notes the maximum of its logits of each tile.
// The K-th largest maximum of groups of threads is then a bound that at least K logits reach and, the
// groups being a random partition as it were, not many more; they stand where the noted maxima reach it, and
// those few places are read again.  The loop has neither barriers nor shared counters (collecting
// candidates in it took 34 us for 256 rows of 131072 bf16 logits, of which streaming alone is 14.4).
// Where more logits reach the bound than there is room for (equal ones, or few groups that have nearly all), the
// bound is raised by those that were kept, twice at most; the K-th largest of what may still be too many (fewer
// groups than K have thousands of the largest) is found by bisection.
//
// s is formed as an unevaluated sum of two fp32 numbers and rounded to fp32 once.  Their order within a row, and that
// of equal rows, is exact; between rows L is as good as its sum, which is fp32: off by 4.2e-6 at most, counting
// roundings (rows of up to 160000 logits), and with that last rounding by up to 7e-7 where it was measured (logits
// of spread 1 to 10, six shapes).
#include "branch.h"

#include <cooperative_groups.h>
#include <cstring>
#include <type_traits>

namespace fa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = kBeamThreads;
constexpr int kCap = 512;                     // candidates that there is room for
constexpr int kJoinCap = 1024;
constexpr int kJoinOwn = 4;                   // a thread's candidates that stay in registers
constexpr int kPlaces = 64;                   // of a warp's list
constexpr float kLog2e = 1.4426950408889634f;
constexpr unsigned kAll = 0xffffffffu;

// An order-preserving map of floats to unsigned integers (-0 as +0); 0 stands for none.
__device__ __forceinline__ unsigned order_of(float x) {
    const unsigned u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned u) {
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
// Lanes that share the work on one of n things (a power of two up to 32).
template <int THREADS>
__device__ __forceinline__ int lanes_each(int n) {
    int p = 32;
    while (p > 1 && n * p > THREADS) p /= 2;
    return p;
}
__device__ __forceinline__ int sum_lanes(int x, int p) {
    for (int o = p / 2; o > 0; o /= 2) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

// The k-th largest of values[0 .. n), n a power of two from 32 to the CTA's threads: the largest that k of them
// reach.  Every thread calls it and gets the result; *out has to be 0 before.
template <int THREADS>
__device__ __forceinline__ unsigned kth_largest(const unsigned *values, int n, int k, unsigned *out) {
    const uint4 *fours = reinterpret_cast<const uint4 *>(values);
    if (n == 32) {  // every warp for itself
        const unsigned mine = values[lane_id()];
        int reached = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint4 x = fours[j];
            reached += (x.x >= mine) + (x.y >= mine) + (x.z >= mine) + (x.w >= mine);
        }
        return __reduce_max_sync(kAll, reached >= k ? mine : 0);
    }
    const int lanes = min(lanes_each<THREADS>(n), n / 4), part = threadIdx.x % lanes;
    const int i = static_cast<int>(threadIdx.x) / lanes;
    if (i < n) {  // whole warps
        const unsigned mine = values[i];
        int reached = 0;
#pragma unroll 4
        for (int j = part; j < n / 4; j += lanes) {
            const uint4 x = fours[j];
            reached += (x.x >= mine) + (x.y >= mine) + (x.z >= mine) + (x.w >= mine);
        }
        reached = sum_lanes(reached, lanes);
        const unsigned best = __reduce_max_sync(kAll, reached >= k ? mine : 0);
        if (lane_id() == 0) atomicMax(out, best);
    }
    __syncthreads();
    return *out;
}

// Groups whose maxima bound the K largest.
__device__ __forceinline__ int group_count(int K) { return K <= 16 ? 32 : K <= 32 ? 64 : K <= 64 ? 128 : 256; }

// The sum of x over the CTA's threads, the same in each; `scratch` holds a word per warp.
template <int THREADS = kThreads>
__device__ __forceinline__ int block_sum(int x, int *scratch) {
    x = __reduce_add_sync(kAll, x);
    __syncthreads();
    if (lane_id() == 0) scratch[warp_id()] = x;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) s += scratch[w];
    return s;
}

template <int BYTES>
struct VecOf;
template <> struct VecOf<16> { using type = uint4; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<4> { using type = unsigned; };
template <> struct VecOf<2> { using type = unsigned short; };

template <int TYPE>
using beam_elem = typename std::conditional<TYPE == kBeamF32, float,
                                            typename std::conditional<TYPE == kBeamBF16, __nv_bfloat16,
                                                                      __half>::type>::type;

template <int TYPE>
__device__ __forceinline__ float beam_float(beam_elem<TYPE> x) {
    if constexpr (TYPE == kBeamF32) return x;
    else if constexpr (TYPE == kBeamBF16) return __bfloat162float(x);
    else return __half2float(x);
}

// A thread's logits of a tile as they were loaded.  Logit i * VEC + k of the thread is number
// (i * THREADS + tid) * VEC + k of the tile; behind the row's end they are -inf.
template <int TYPE, int VEC, int THREADS>
struct BeamTile {
    using Elem = beam_elem<TYPE>;
    using Vec = typename VecOf<VEC * sizeof(Elem)>::type;
    static constexpr int kElems = beam_elems(TYPE, VEC), kSize = kElems * THREADS;
    Vec raw[kElems / VEC];

    static __device__ __forceinline__ int place(int e, int tid = threadIdx.x) {
        return (e / VEC * THREADS + tid) * VEC + e % VEC;
    }
    // x: the tile's first logit; left: how many there are to the end
    __device__ __forceinline__ void load(const Elem *x, int left) {
        if (left >= kSize) {
            const Vec *from = reinterpret_cast<const Vec *>(x) + threadIdx.x;
#pragma unroll
            for (int i = 0; i < kElems / VEC; ++i) raw[i] = __ldcs(from + i * THREADS);
            return;
        }
#pragma unroll
        for (int i = 0; i < kElems / VEC; ++i) {
            const int at = place(i * VEC);
            Elem e[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                if (at + k < left) e[k] = x[at + k];
                else if constexpr (TYPE == kBeamF32) e[k] = -INFINITY;
                else if constexpr (TYPE == kBeamBF16) e[k] = __ushort_as_bfloat16(0xff80);
                else e[k] = __ushort_as_half(0xfc00);
            }
            memcpy(&raw[i], e, sizeof(Vec));
        }
    }
    __device__ __forceinline__ void floats(float (&v)[kElems]) const {
        if constexpr (TYPE != kBeamF32 && VEC > 1) {
            uint32_t word[kElems / 2];
            memcpy(word, raw, sizeof(raw));
#pragma unroll
            for (int k = 0; k < kElems / 2; ++k) {
                if constexpr (TYPE == kBeamBF16) {  // one instruction each
                    v[2 * k] = __uint_as_float(word[k] << 16);
                    v[2 * k + 1] = __uint_as_float(word[k] & 0xffff0000u);
                } else {
                    const float2 f = unpack2<false>(word[k]);
                    v[2 * k] = f.x, v[2 * k + 1] = f.y;
                }
            }
        } else {
            const Elem *e = reinterpret_cast<const Elem *>(raw);
#pragma unroll
            for (int k = 0; k < kElems; ++k) v[k] = beam_float<TYPE>(e[k]);
        }
    }
};

// The CTA's work on one piece of a row: its K best into keys, its sum into *stats.
template <int TYPE, int VEC, int THREADS>
__device__ __forceinline__ void beam_piece(const BeamParams &p, int row, int piece,
                                           unsigned long long *keys, float2 *stats) {
    using Tile = BeamTile<TYPE, VEC, THREADS>;
    using Elem = typename Tile::Elem;
    constexpr int kElems = Tile::kElems;
    __shared__ float tops[kBeamNoted / THREADS][THREADS];  // of each thread's logits of each tile
    __shared__ __align__(16) unsigned groups[256];
    __shared__ unsigned bound;
    __shared__ int found;
    __shared__ int scratch[THREADS / 32];
    __shared__ unsigned tops_of[THREADS / 32];  // each warp's maximum
    __shared__ unsigned short places[THREADS / 32][kPlaces];
    __shared__ float sums[THREADS / 32];
    __shared__ unsigned long long cand[kCap];
    static_assert(kCap == 2 * THREADS && THREADS == 256);
    const int tid = threadIdx.x, lane = lane_id();
    const int b = row / p.W, w = row - b * p.W;
    const int v0 = piece * p.piece_len, len = min(p.V - v0, p.piece_len);
    const Elem *x = static_cast<const Elem *>(p.logits) + b * p.stride_b + w * p.stride_w + v0;
    const int K = p.K;
    const int tiles = (len - 1) / Tile::kSize + 1;
    float m = -INFINITY, s = 0.f;  // this thread's maximum, and sum of e^(x - m)
    Tile next;
    next.load(x, len);
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
        float v[kElems];
        next.floats(v);
        const int after = (t + 1) * Tile::kSize;
        if (t + 1 < tiles) next.load(x + after, len - after);
        float a = fmax3(v[0], v[1], v[2]), c = fmax3(v[3], v[4], v[5]);
#pragma unroll
        for (int e = 6; e + 3 < kElems; e += 4) {
            a = fmax3(a, v[e], v[e + 1]);
            c = fmax3(c, v[e + 2], v[e + 3]);
        }
        const float top = fmax3(fmaxf(a, c), v[kElems - 2], v[kElems - 1]);
        tops[t][tid] = top;
        if (top > m) {
            s *= ex2((m - top) * kLog2e);
            m = top;
        }
        const float ref = m == -INFINITY ? 0.f : m;  // nothing but -inf so far sums to 0
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f)};
#pragma unroll
        for (int e = 0; e < kElems; e += 2) {
            // the difference first: its rounding is relative to itself, and 0 for the largest
            const float2 y = fmul2(fsub2(make_float2(v[e], v[e + 1]), make_float2(ref, ref)),
                                   make_float2(kLog2e, kLog2e));
            acc[e / 2 & 3] = fadd2(acc[e / 2 & 3], make_float2(ex2(y.x), ex2(y.y)));
        }
        const float2 q = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
        s += q.x + q.y;
    }

    // groups of threads, at least twice as many as wanted
    const int count = group_count(K), width = THREADS / count;
    float g = m;
    for (int o = 1; o < width; o *= 2) g = fmaxf(g, __shfl_xor_sync(kAll, g, o));
    if (tid % width == 0) groups[tid / width] = order_of(g);
    const unsigned mine = __reduce_max_sync(kAll, order_of(m));
    if (lane == 0) tops_of[warp_id()] = mine;
    if (tid == 0) found = 0, bound = 0;
    __syncthreads();
    unsigned least = kth_largest<THREADS>(groups, count, K, &bound);  // K logits at least reach it
    unsigned most = tops_of[0];
#pragma unroll
    for (int i = 1; i < THREADS / 32; ++i) most = max(most, tops_of[i]);
    const float top = value_of(most);
    if (m != -INFINITY) s *= ex2((m - top) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if (lane == 0) sums[warp_id()] = s;
    auto key_of = [&](float v, int place) {  // larger: a larger logit, or the first of equal ones
        return static_cast<unsigned long long>(order_of(v)) << 32 | ~static_cast<unsigned>(v0 + place);
    };
    auto take = [&](float v, int place) {
        const int at = atomicAdd(&found, 1);
        if (at < kCap) cand[at] = key_of(v, place);
    };
    // First the logits that reach the bound: what is above the next lower number (below +0 that is not -0; -inf is
    // never a candidate).  Where these are too many, a few groups having most of what is to be had, those that were
    // kept are a sample of them: the K-th largest of its pairs' maxima is the next bound, and the logits above that
    // are collected, or those above the bound that was, where too few pairs exceed it.  (256 rows of 131072 bf16
    // logits, all but a run of 1000 masked, K 64: 41 us, 177 by bisection at once; 80 rows of 50000, the last 848
    // logits a piece's last, K 16: 23 and 49.)
    float over = least <= order_of(-INFINITY) ? -INFINITY : value_of(least - (least == 0x80000000u ? 2 : 1));
    int n = 0, pass = 0;
#pragma unroll 1
    for (;; ++pass) {
        // The threads' tiles that have a logit to collect are listed and read again by the warp, a logit per
        // lane, eight reads in flight.
        if (__any_sync(kAll, m > over)) {
            unsigned short *list = places[warp_id()];
            int listed = 0;
            for (int t = 0; t <= tiles; ++t) {
                const unsigned who = __ballot_sync(kAll, t < tiles && tops[t < tiles ? t : 0][tid] > over);
                if (t == tiles || listed + __popc(who) > kPlaces) {
                    constexpr int kAtOnce = 32 / kElems, kBatch = 8;
                    __syncwarp();
                    auto full = [&] { return *static_cast<volatile int *>(&found) > kCap; };
                    for (int i0 = lane / kElems; i0 < listed && !full(); i0 += kAtOnce * kBatch) {
                        float v[kBatch];
                        int at[kBatch];
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            v[k] = -INFINITY;
                            if (i0 + k * kAtOnce >= listed) continue;
                            const int from = list[i0 + k * kAtOnce];
                            at[k] = from / 32 * Tile::kSize + Tile::place(lane % kElems, (tid & ~31) + from % 32);
                            if (at[k] < len) v[k] = beam_float<TYPE>(x[at[k]]);
                        }
#pragma unroll
                        for (int k = 0; k < kBatch; ++k)
                            if (v[k] > over) take(v[k], at[k]);
                    }
                    __syncwarp();
                    listed = 0;
                    if (__any_sync(kAll, full())) break;
                }
                if (who >> lane & 1)
                    list[listed + __popc(who & ((1u << lane) - 1))] = static_cast<unsigned short>(32 * t + lane);
                listed += __popc(who);
            }
        }
        __syncthreads();
        n = found;
        if (n <= kCap || pass == 2) break;
        const unsigned pair = static_cast<unsigned>(max(cand[tid], cand[tid + THREADS]) >> 32);
        groups[tid] = pair;
        const int above = __syncthreads_count(pair > least);
        if (tid == 0) found = 0, bound = 0;
        __syncthreads();
        if (above >= K) least = kth_largest<THREADS>(groups, THREADS, K, &bound);
        over = value_of(least);
    }
    if (pass > 0) {
        // Too many reached the first bound.  f(logit, its place in the piece) for this thread's logits of tiles
        // that have one of that order or a higher one
        auto each = [&](unsigned want, auto f) {
            for (int t = 0; t < tiles; ++t) {
                if (!(order_of(tops[t][tid]) >= want)) continue;
#pragma unroll 1
                for (int i = 0; i < kElems / VEC; ++i) {
                    const int at = t * Tile::kSize + Tile::place(i * VEC);
                    for (int k = 0; k < VEC && at + k < len; ++k) f(beam_float<TYPE>(x[at + k]), at + k);
                }
            }
        };
        auto reach = [&](unsigned want) {
            int c = 0;
            each(want, [&](float v, int) { c += v > -INFINITY && order_of(v) >= want; });
            return block_sum<THREADS>(c, scratch);
        };
        unsigned lo = least;  // the K-th largest: the bound, or, where too many are above it too, found by bisection
        if (n > kCap) {
            unsigned hi = ~0u;
            while (hi - lo > 1) {
                const unsigned mid = lo + (hi - lo) / 2;
                if (reach(mid) >= K) lo = mid;
                else hi = mid;
            }
            if (tid == 0) found = 0;
            __syncthreads();
            each(lo + 1, [&](float v, int place) {
                if (order_of(v) > lo && v > -INFINITY) take(v, place);
            });
            __syncthreads();
            n = found;
        }
        // of its equals, the first that make K: up to place `end`
        const int room = K - n;
        const float equal = value_of(lo);
        if (room > 0) {
            auto equals = [&](int from, int to) {
                int c = 0;
#pragma unroll 8
                for (int i = from + tid; i < min(to, len); i += THREADS) c += beam_float<TYPE>(x[i]) == equal;
                return block_sum<THREADS>(c, scratch);
            };
            int end = 0, before = 0;
            for (int span = 8 * THREADS; end < len;) {
                const int c = equals(end, end + span);
                if (before + c < room) before += c, end += span;
                else if (span == 1) break;
                else span /= 2;
            }
            for (int i = tid; i < min(end + 1, len); i += THREADS)
                if (beam_float<TYPE>(x[i]) == equal) take(equal, i);
            __syncthreads();
            n = found;
        }
    }
    // the K largest, largest first, by counting: a warp's work where there are few
    const int lanes = n <= 32 ? 1 : lanes_each<THREADS>(n), part = tid & (lanes - 1), own = tid / lanes;
    for (int i0 = 0; i0 + (tid & ~31) / lanes < n; i0 += THREADS / lanes) {  // whole warps
        const int i = i0 + own;
        const unsigned long long k = i < n ? cand[i] : 0;
        int rank = 0;
#pragma unroll 4
        for (int j = part; j < n; j += lanes) rank += cand[j] > k;
        rank = sum_lanes(rank, lanes);
        if (i < n && part == 0 && rank < K) keys[rank] = k;
    }
    for (int i = n + tid; i < K; i += THREADS) keys[i] = 0;
    if (tid == THREADS - 1) {
        float sum = sums[0];
#pragma unroll
        for (int i = 1; i < THREADS / 32; ++i) sum += sums[i];
        *stats = make_float2(top, sum);
    }
}

// VEC: logits per load, what the rows' alignment allows.
template <int TYPE, int VEC>
__global__ void __launch_bounds__(kThreads, 4) fa_beam_piece_kernel(const BeamParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int row = blockIdx.x / p.pieces, piece = blockIdx.x - row * p.pieces;
    if (p.finished != nullptr && p.finished[row] != 0) return;
    const long out = static_cast<long>(row) * p.pieces + piece;
    beam_piece<TYPE, VEC, kThreads>(p, row, piece, p.keys + out * p.K, p.stats + out);
}

// hi + lo, in order as unsigned integers: lo is what hi's rounding left.  0 where it is not finite.
__device__ __forceinline__ unsigned long long pair_order(float hi, float lo) {
    return fabsf(hi) < INFINITY ? static_cast<unsigned long long>(order_of(hi)) << 32 | order_of(lo) : 0;
}
// a + b and what its rounding left.
__device__ __forceinline__ float2 two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}

// ln s as a pair, reduced after Cody and Waite: the exponent's share is exact to 2^-36 (the first term of ln 2 has
// 12 bits), that of the mantissa off by a rounding of a value below 0.7.
__device__ __forceinline__ float2 pair_log(float s) {
    int e;
    const float f = frexpf(s, &e);
    const float2 r = two_sum(e * 0.693115234375f, logf(f));
    return make_float2(r.x, fmaf(static_cast<float>(e), 3.1946184945309417e-05f, r.y));
}

// What a request's beams add to a logit: (hi, lo) of score - ln of the beam's sum (NaN: it offers nothing),
// and the maximum that the sum refers to.  They are kept apart: x less the maximum is exact as a pair,
// whatever their size.
struct BeamBase {
    float hi, lo, ref;
    int ended;  // the beam has one candidate, the end token at score hi
};

// One CTA joins the pieces of request b: the sums, then the K best candidates, by a bound and counting as for
// the pieces.  A request has up to a few thousand candidates and the time is that of the chain of steps,
// so many threads share each count.  list_of(l) and stats_of(l): the candidates and the sum of
// piece l % pieces of beam l / pieces.
template <int THREADS, class Lists, class Stats>
__device__ __forceinline__ void beam_join(const BeamParams &p, int b, BeamBase *base, Lists list_of,
                                          Stats stats_of) {
    __shared__ __align__(16) unsigned groups[256];
    __shared__ unsigned bound;
    __shared__ int found;
    __shared__ int scratch[THREADS / 32];
    __shared__ unsigned long long cand[kJoinCap];
    __shared__ int where[kJoinCap];
    const int tid = threadIdx.x, lane = lane_id();
    const int W = p.W, K = p.K, S = p.pieces, V = p.V;
    const uint8_t *finished = p.finished != nullptr ? p.finished + static_cast<long>(b) * W : nullptr;
    // `lanes` threads take a list, each every lanes-th of its candidates; a thread's first ones stay in registers
    int lanes = 1;
    while (lanes < K && lanes < 32) lanes *= 2;
    const int part = tid % lanes, each_turn = THREADS / lanes, lists = W * S;
    const int deep = (K + lanes - 1) / lanes;  // candidates of a list for each thread
    unsigned long long own[kJoinOwn];
    int l0 = tid / lanes, d0 = 0;  // where the thread's candidates go on behind the registers
#pragma unroll
    for (int r = 0; r < kJoinOwn; ++r) {
        const int j = part + d0 * lanes;
        own[r] = l0 < lists && j < K && (finished == nullptr || finished[l0 / S] == 0) ? list_of(l0)[j] : 0;
        if (++d0 == deep) d0 = 0, l0 += each_turn;
    }
    for (int w = warp_id(); w < W; w += THREADS / 32) {
        const float score = p.scores[static_cast<long>(b) * W + w];
        if (finished != nullptr && finished[w] != 0) {
            if (lane == 0) base[w] = {score, 0.f, 0.f, 1};
            continue;
        }
        float m = -INFINITY;
        for (int i = lane; i < S; i += 32) m = fmaxf(m, stats_of(w * S + i).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        float s = 0.f;
        for (int i = lane; i < S; i += 32) {
            const float2 st = stats_of(w * S + i);
            s += st.x == -INFINITY ? st.y : st.y * ex2((st.x - m) * kLog2e);  // y: 0 or NaN
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        if (lane == 0) {
            const float2 l = pair_log(s), r = two_sum(score, -l.x);
            // nothing to choose from, or a logit that is no number
            const bool none = !(m > -INFINITY && s < INFINITY);
            base[w] = {none ? NAN : r.x, r.y - l.y, m, 0};
        }
    }
    if (tid == 0) found = 0, bound = 0;
    if (tid < 256) groups[tid] = 0;
    __syncthreads();
    // the order (0: none) of candidate j of list l, whose key is k, and its place w V + v
    auto order = [&](int l, int j, unsigned long long k, int *at) -> unsigned long long {
        const int w = l / S;
        const BeamBase c = base[w];
        if (c.ended) {
            *at = w * V + p.end_token;
            return l == w * S && j == 0 ? pair_order(c.hi, 0.f) : 0;
        }
        if (k == 0) return 0;
        *at = w * V + static_cast<int>(~static_cast<unsigned>(k));
        const float2 d = two_sum(value_of(static_cast<unsigned>(k >> 32)), -c.ref);
        const float2 s = two_sum(d.x, c.hi);
        const float2 r = two_sum(s.x, s.y + (d.y + c.lo));
        return pair_order(r.x, r.y);
    };
    // K candidates at least reach the K-th largest of the best ones of groups, to which they go scattered
    const int count = group_count(K);
    int place[kJoinOwn];
    {
        int l = tid / lanes, d = 0;
#pragma unroll
        for (int r = 0; r < kJoinOwn; ++r) {
            const int j = part + d * lanes;
            place[r] = 0;
            own[r] = l < lists && j < K ? order(l, j, own[r], &place[r]) : 0;
            if (own[r] != 0) atomicMax(&groups[(37 * l + 11 * j) % count], static_cast<unsigned>(own[r] >> 32));
            if (++d == deep) d = 0, l += each_turn;
        }
    }
    // f(order, place) for this thread's candidates from behind the registers on
    auto rest = [&](auto f) {
        for (int l = l0, d = d0; l < lists; l += each_turn, d = 0)
            for (; d < deep; ++d) {
                const int j = part + d * lanes;
                if (j >= K) continue;
                int at = 0;
                const unsigned long long k = order(l, j, base[l / S].ended ? 0 : list_of(l)[j], &at);
                f(k, at, 37 * l + 11 * j);
            }
    };
    rest([&](unsigned long long k, int, int group) {
        if (k != 0) atomicMax(&groups[group % count], static_cast<unsigned>(k >> 32));
    });
    auto each = [&](auto f) {
#pragma unroll
        for (int r = 0; r < kJoinOwn; ++r) f(own[r], place[r]);
        rest([&](unsigned long long k, int at, int) { f(k, at); });
    };
    auto take = [&](unsigned long long k, int at) {
        const int n = atomicAdd(&found, 1);
        if (n < kJoinCap) cand[n] = k, where[n] = at;
    };
    __syncthreads();
    const unsigned least = kth_largest<THREADS>(groups, count, K, &bound);
    const unsigned long long t = max(static_cast<unsigned long long>(least) << 32, 1ull);
    each([&](unsigned long long k, int at) {
        if (k >= t) take(k, at);
    });
    __syncthreads();
    int n = found;
    if (n > kJoinCap) {
        // The K-th best by bisection on the score, then on the place of its equals.
        unsigned long long lo = t, hi = ~0ull;  // lo is reached by K or more
        auto reach = [&](auto test) {
            int c = 0;
            each([&](unsigned long long k, int at) { c += test(k, at); });
            return block_sum<THREADS>(c, scratch);
        };
        while (hi - lo > 1) {
            const unsigned long long mid = lo + (hi - lo) / 2;
            if (reach([&](unsigned long long k, int) { return k >= mid; }) >= K) lo = mid;
            else hi = mid;
        }
        const int room = K - reach([&](unsigned long long k, int) { return k > lo; });
        int end = 0;  // the place of the last of the equals that are taken
#pragma unroll 1
        for (int bit = 30; bit >= 0; --bit) {
            const int to = end | 1 << bit;
            if (reach([&](unsigned long long k, int at) { return k == lo && at < to; }) < room) end = to;
        }
        if (tid == 0) found = 0;
        __syncthreads();
        each([&](unsigned long long k, int at) {
            if (k > lo || (k == lo && at <= end)) take(k, at);
        });
        __syncthreads();
        n = found;
    }
    const long out = static_cast<long>(b) * K;
    const int share = lanes_each<THREADS>(n), turn = tid % share;
    for (int i0 = 0; i0 < n; i0 += THREADS / share) {
        const int i = i0 + tid / share;
        const bool there = i < n;
        if (!__any_sync(kAll, there)) continue;
        const unsigned long long mine = there ? cand[i] : 0;
        const int spot = there ? where[i] : 0;
        int rank = 0;
#pragma unroll 4
        for (int j = turn; j < n; j += share) {
            const unsigned long long other = cand[j];
            const int at = where[j];  // read in any case: nothing waits for the comparison
            rank += other > mine || (other == mine && at < spot);
        }
        rank = sum_lanes(rank, share);
        if (there && turn == 0 && rank < K) {
            const int w = spot / V, v = spot - w * V;
            p.out_scores[out + rank] = value_of(static_cast<unsigned>(mine >> 32));
            p.parents[out + rank] = b * W + w;
            p.tokens[out + rank] = v;
            p.out_finished[out + rank] = v == p.end_token || base[w].ended != 0;
        }
    }
    for (int k = n + tid; k < K; k += THREADS) {
        p.out_scores[out + k] = -INFINITY;
        p.parents[out + k] = p.tokens[out + k] = -1;
        p.out_finished[out + k] = 1;
    }
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) fa_beam_join_kernel(const BeamParams p) {
    extern __shared__ BeamBase base[];  // [W]
    griddep_launch_dependents();
    griddep_wait();
    const long first = static_cast<long>(blockIdx.x) * p.W * p.pieces;  // of the request's pieces
    beam_join<THREADS>(
        p, blockIdx.x, base, [&](int l) { return p.keys + (first + l) * p.K; },
        [&](int l) { return p.stats[first + l]; });
}

// Small requests in one launch, without a workspace: a cluster per request, whose CTAs take pieces in turns
// and leave lists and sums in their shared memory, where the first CTA reads them.
template <int TYPE, int VEC>
__global__ void __launch_bounds__(kThreads, 2) fa_beam_cluster_kernel(const BeamParams p) {
    extern __shared__ __align__(16) unsigned char beam_smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int cta = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
    const int units = p.W * p.pieces, slots = (units + ctas - 1) / ctas;
    unsigned long long *lists = reinterpret_cast<unsigned long long *>(beam_smem);  // [slots][K]
    float2 *stats = reinterpret_cast<float2 *>(lists + slots * p.K);                // [slots]
    BeamBase *base = reinterpret_cast<BeamBase *>(stats + slots);                   // [W]
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x / ctas;
    for (int u = cta, slot = 0; u < units; u += ctas, ++slot) {
        const int w = u / p.pieces, row = b * p.W + w;
        if (p.finished != nullptr && p.finished[row] != 0) continue;
        if (slot > 0) __syncthreads();  // the piece before is out of the way
        beam_piece<TYPE, VEC, kThreads>(p, row, u - w * p.pieces, lists + slot * p.K, stats + slot);
    }
    cluster.sync();
    if (cta == 0)
        beam_join<kThreads>(
            p, b, base, [&](int l) { return cluster.map_shared_rank(lists, l % ctas) + l / ctas * p.K; },
            [&](int l) { return cluster.map_shared_rank(stats, l % ctas)[l / ctas]; });
    cluster.sync();  // the lists have been read
}

template <int TYPE, int VEC>
cudaError_t launch_vec(const BeamParams &p, cudaStream_t stream) {
    if (p.ctas == 0) {
        const cudaError_t e = launch_overlapped(fa_beam_piece_kernel<TYPE, VEC>, dim3(p.pieces * p.B * p.W),
                                                kThreads, 0, stream, p);
        if (e != cudaSuccess) return e;
        // few candidates: many small CTAs instead of ones that take half an SM each
        const size_t smem = sizeof(BeamBase) * p.W;
        return static_cast<long>(p.W) * p.pieces * p.K <= 4 * kThreads
                   ? launch_overlapped(fa_beam_join_kernel<kThreads>, dim3(p.B), kThreads, smem, stream, p)
                   : launch_overlapped(fa_beam_join_kernel<1024>, dim3(p.B), 1024, smem, stream, p);
    }
    const int slots = (p.W * p.pieces + p.ctas - 1) / p.ctas;
    // 128 pieces in 16 CTAs: 10 KB at most, beside 36
    const size_t smem = slots * (p.K * sizeof(unsigned long long) + sizeof(float2)) + p.W * sizeof(BeamBase);
    return launch_clusters(fa_beam_cluster_kernel<TYPE, VEC>, p.B, p.ctas, kThreads, smem, stream, p);
}

template <int TYPE>
cudaError_t launch_type(const BeamParams &p, int vec, cudaStream_t stream) {
    if constexpr (TYPE != kBeamF32)
        if (vec == 8) return launch_vec<TYPE, 8>(p, stream);
    return vec == 4 ? launch_vec<TYPE, 4>(p, stream)
           : vec == 2 ? launch_vec<TYPE, 2>(p, stream)
                      : launch_vec<TYPE, 1>(p, stream);
}

}  // namespace

cudaError_t launch_beam_select(const BeamParams &p, int type, int vec, cudaStream_t stream) {
    return type == kBeamF32    ? launch_type<kBeamF32>(p, vec, stream)
           : type == kBeamBF16 ? launch_type<kBeamBF16>(p, vec, stream)
                               : launch_type<kBeamF16>(p, vec, stream);
}

}  // namespace fa
