// fa_beam.cu - beam search's selection over beams and vocabulary.
//
// Candidate (w, v) of a request continues beam w with token v and scores
//   s(w, v) = score_w + x_wv - L_w,   L_w = ln sum_v e^x_wv,
// and the K best of the W V candidates are wanted, equal ones by the lowest w V + v.  Within a row the
// order of s is that of x, so a row's logits are read once: a CTA takes a piece of a row into
// registers, finds its maximum m and sum of e^(x - m) (fp32; the maximum is known before the first
// exponential) and its K largest x; a second, small grid joins the pieces' statistics and candidates of
// a request.  Bound by reading the logits from HBM.
//
// The K largest of a piece: the K-th largest of the maxima of 64 (or 256) groups of its logits is a
// bound that at least K logits reach and, the groups being a random partition as it were, not many
// more.  Those that reach it are collected and ranked by counting.  Where too many do (a piece of
// equal logits), the K-th largest is found by bisection, first on the value, then on the place.
//
// s is formed in 64 bits from the fp32 sums, so candidates of different beams are told apart well below
// the fp32 spacing of the scores, to which the result is rounded once.
#include "branch.h"

#include <type_traits>

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kElems = kBeamChunk / kThreads;  // logits of a thread
constexpr int kCap = 1024;                     // candidates that are ranked by counting
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
__device__ __forceinline__ unsigned long long order_of(double x) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
    return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double value_of(unsigned long long u) {
    return __longlong_as_double(static_cast<long long>(u >> 63 ? u ^ 1ull << 63 : ~u));
}

// The k-th largest of the warp's 32 * N values (k at most that many), by bits from the top.
template <int N>
__device__ __forceinline__ unsigned kth_largest(const unsigned (&v)[N], int k) {
    unsigned found = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
        const unsigned want = found | 1u << bit;
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) n += __popc(__ballot_sync(kAll, v[i] >= want));
        if (n >= k) found = want;
    }
    return found;
}

// The sum of x over the CTA's threads, the same in each; `scratch` holds a word per warp.
__device__ __forceinline__ int block_sum(int x, int *scratch) {
    x = __reduce_add_sync(kAll, x);
    __syncthreads();
    if (lane_id() == 0) scratch[warp_id()] = x;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += scratch[w];
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

// VEC: logits per load, what the rows' alignment allows.
template <int TYPE, int VEC>
__global__ void __launch_bounds__(kThreads) fa_beam_piece_kernel(const BeamParams p) {
    using Elem = beam_elem<TYPE>;
    using Vec = typename VecOf<VEC * sizeof(Elem)>::type;
    __shared__ unsigned groups[kThreads];
    __shared__ unsigned bound;
    __shared__ int found;
    __shared__ int scratch[kThreads / 32];
    __shared__ float sums[kThreads / 32];
    __shared__ unsigned long long cand[kCap];
    griddep_launch_dependents();
    griddep_wait();
    const int row = blockIdx.x / p.chunks, piece = blockIdx.x - row * p.chunks;
    const int tid = threadIdx.x, lane = lane_id();
    if (p.finished != nullptr && p.finished[row] != 0) return;
    const int b = row / p.W, w = row - b * p.W;
    const int v0 = piece * kBeamChunk, left = p.V - v0;
    const Elem *x = static_cast<const Elem *>(p.logits) + b * p.stride_b + w * p.stride_w + v0;

    // logit i * VEC + k of the thread is number (i * kThreads + tid) * VEC + k of the piece
    float v[kElems];
    auto place = [&](int e) { return (e / VEC * kThreads + tid) * VEC + e % VEC; };
    Vec raw[kElems / VEC];
#pragma unroll
    for (int i = 0; i < kElems / VEC; ++i) {
        if ((i * kThreads + tid) * VEC + VEC <= left)
            raw[i] = __ldcs(reinterpret_cast<const Vec *>(x) + i * kThreads + tid);
    }
#pragma unroll
    for (int i = 0; i < kElems / VEC; ++i) {
        const int at = (i * kThreads + tid) * VEC;
        const Elem *e = reinterpret_cast<const Elem *>(&raw[i]);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            if (at + VEC <= left) v[i * VEC + k] = beam_float<TYPE>(e[k]);
            else v[i * VEC + k] = at + k < left ? beam_float<TYPE>(x[at + k]) : -INFINITY;
        }
    }
    float top = v[0];
#pragma unroll
    for (int e = 1; e < kElems; ++e) top = fmaxf(top, v[e]);
    // groups of four threads up to K = 64, of one behind that
    const bool wide = p.K > 64;
    const float four = fmaxf(fmaxf(top, __shfl_xor_sync(kAll, top, 1)),
                             __shfl_xor_sync(kAll, fmaxf(top, __shfl_xor_sync(kAll, top, 1)), 2));
    if (wide) groups[tid] = order_of(top);
    else if ((lane & 3) == 0) groups[tid / 4] = order_of(four);
    if (tid == 0) found = 0;
    __syncthreads();
    unsigned most = 0;
    if (wide) {
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) most = max(most, groups[lane + 32 * i]);
    } else {
        most = max(groups[lane], groups[lane + 32]);
    }
    most = __reduce_max_sync(kAll, most);
    if (warp_id() == 0) {
        unsigned t;
        if (wide) {
            unsigned g[kThreads / 32];
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) g[i] = groups[lane + 32 * i];
            t = kth_largest(g, p.K);
        } else {
            const unsigned g[2] = {groups[lane], groups[lane + 32]};
            t = kth_largest(g, p.K);
        }
        if (lane == 0) bound = t;
    }
    const float m = value_of(most);
    const float ref = m == -INFINITY ? 0.f : m;  // a piece of nothing but -inf sums to 0
    float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                     make_float2(0.f, 0.f)};
#pragma unroll
    for (int e = 0; e < kElems; e += 2) {
        // the difference first: its rounding is relative to itself, and 0 for the largest
        const float2 y = fmul2(fsub2(make_float2(v[e], v[e + 1]), make_float2(ref, ref)),
                               make_float2(kLog2e, kLog2e));
        acc[e / 2 & 3] = fadd2(acc[e / 2 & 3], make_float2(ex2(y.x), ex2(y.y)));
    }
    const float2 a = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
    float sum = a.x + a.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (lane == 0) sums[warp_id()] = sum;
    __syncthreads();
    const float t = value_of(bound);
    auto key = [&](int e) {
        return static_cast<unsigned long long>(order_of(v[e])) << 32 | ~static_cast<unsigned>(v0 + place(e));
    };
    if (top >= t) {
#pragma unroll
        for (int e = 0; e < kElems; ++e)
            if (v[e] >= t && v[e] > -INFINITY) {
                const int at = atomicAdd(&found, 1);
                if (at < kCap) cand[at] = key(e);
            }
    }
    __syncthreads();
    int n = found;
    if (n > kCap) {
        // rare: the K-th largest by bisection on the value, then on the place of its equals
        unsigned lo = 0;
#pragma unroll 1
        for (int bit = 31; bit >= 0; --bit) {
            const unsigned want = lo | 1u << bit;
            int c = 0;
#pragma unroll
            for (int e = 0; e < kElems; ++e) c += v[e] > -INFINITY && order_of(v[e]) >= want;
            if (block_sum(c, scratch) >= p.K) lo = want;
        }
        int above = 0;
#pragma unroll
        for (int e = 0; e < kElems; ++e) above += v[e] > -INFINITY && order_of(v[e]) > lo;
        const int room = p.K - block_sum(above, scratch);
        int end = 0;  // the first places up to which fewer than `room` of the equals lie
#pragma unroll 1
        for (int bit = kBeamChunk / 2; bit > 0; bit /= 2) {
            int c = 0;
#pragma unroll
            for (int e = 0; e < kElems; ++e) c += order_of(v[e]) == lo && place(e) < end + bit;
            if (block_sum(c, scratch) < room) end += bit;
        }
        if (tid == 0) found = 0;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kElems; ++e) {
            const unsigned o = order_of(v[e]);
            if (v[e] > -INFINITY && (o > lo || (o == lo && place(e) <= end)))
                cand[atomicAdd(&found, 1)] = key(e);
        }
        __syncthreads();
        n = found;
    }
    const long out = static_cast<long>(row) * p.chunks + piece;
    unsigned long long *keys = p.keys + out * p.K;
    for (int i = tid; i < n; i += kThreads) {
        const unsigned long long mine = cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += cand[j] > mine;
        if (rank < p.K) keys[rank] = mine;
    }
    for (int i = n + tid; i < p.K; i += kThreads) keys[i] = 0;
    if (tid == 0) {
        float s = sums[0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) s += sums[i];
        p.stats[out] = make_float2(m, s);
    }
}

// ln s in 64 bits: the exponent's share is exact to them, that of the mantissa off by an fp32 rounding
// of a value below 0.7.
__device__ __forceinline__ double wide_log(float s) {
    int e;
    const float f = frexpf(s, &e);
    return e * 0.693147180559945309417 + static_cast<double>(logf(f));
}

// One CTA per request joins its rows' pieces.
__global__ void __launch_bounds__(kThreads) fa_beam_join_kernel(const BeamParams p) {
    // [W] of each beam: score - ln of its sum (NaN for none), and the maximum that the sum refers to.  The
    // two are kept apart: x less the maximum is exact, whatever their size.
    extern __shared__ double base[];
    float *ref = reinterpret_cast<float *>(base + p.W);
    __shared__ unsigned groups[kThreads];
    __shared__ unsigned bound;
    __shared__ int found;
    __shared__ int scratch[kThreads / 32];
    __shared__ unsigned long long cand[kCap];
    __shared__ int where[kCap];
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x, tid = threadIdx.x, lane = lane_id();
    const int W = p.W, K = p.K, S = p.chunks, V = p.V;
    for (int w = warp_id(); w < W; w += kThreads / 32) {
        const int row = b * W + w;
        const double score = static_cast<double>(p.scores[row]);
        if (p.finished != nullptr && p.finished[row] != 0) {
            if (lane == 0) base[w] = score, ref[w] = 0.f;
            continue;
        }
        const float2 *st = p.stats + static_cast<long>(row) * S;
        float m = -INFINITY;
        for (int i = lane; i < S; i += 32) m = fmaxf(m, st[i].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        float s = 0.f;
        for (int i = lane; i < S; i += 32)
            if (st[i].x != -INFINITY) s += st[i].y * ex2((st[i].x - m) * kLog2e);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        if (lane == 0) {
            // nothing to choose from, or a logit that is no number
            base[w] = m > -INFINITY && s < INFINITY ? score - wide_log(s) : __longlong_as_double(-1ll);
            ref[w] = m;
        }
    }
    if (tid == 0) found = 0;
    __syncthreads();
    // candidate i of the request: its order (0: none) and w V + v
    const int list = S * K, total = W * list;
    auto get = [&](int i, int *at) -> unsigned long long {
        const int w = i / list, j = i - w * list, row = b * W + w;
        double s;
        if (p.finished != nullptr && p.finished[row] != 0) {
            if (j != 0) return 0;
            *at = w * V + p.end_token;
            s = base[w];
        } else {
            const unsigned long long k = p.keys[static_cast<long>(row) * list + j];
            if (k == 0) return 0;
            *at = w * V + static_cast<int>(~static_cast<unsigned>(k));
            s = base[w] + (static_cast<double>(value_of(static_cast<unsigned>(k >> 32))) -
                           static_cast<double>(ref[w]));
        }
        return isfinite(s) ? order_of(s) : 0;
    };
    int at = 0;
    unsigned long long most = 0;
    for (int i = tid; i < total; i += kThreads) most = max(most, get(i, &at));
    groups[tid] = static_cast<unsigned>(most >> 32);
    __syncthreads();
    if (warp_id() == 0) {
        unsigned g[kThreads / 32];
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) g[i] = groups[lane + 32 * i];
        const unsigned t = kth_largest(g, K);
        if (lane == 0) bound = t;
    }
    __syncthreads();
    unsigned long long t = static_cast<unsigned long long>(bound) << 32;
    for (int i = tid; i < total; i += kThreads) {
        const unsigned long long k = get(i, &at);
        if (k != 0 && k >= t) {
            const int n = atomicAdd(&found, 1);
            if (n < kCap) cand[n] = k, where[n] = at;
        }
    }
    __syncthreads();
    int n = found;
    if (n > kCap) {
        // rare: the K-th best by bisection on the score, then on the place of its equals
        unsigned long long lo = 0;
#pragma unroll 1
        for (int bit = 63; bit >= 0; --bit) {
            const unsigned long long want = lo | 1ull << bit;
            int c = 0;
            for (int i = tid; i < total; i += kThreads) c += get(i, &at) >= want;
            if (block_sum(c, scratch) >= K) lo = want;
        }
        int above = 0;
        for (int i = tid; i < total; i += kThreads) above += get(i, &at) > lo;
        const int room = K - block_sum(above, scratch);
        int end = 0;
#pragma unroll 1
        for (int bit = 30; bit >= 0; --bit) {
            int c = 0;
            for (int i = tid; i < total; i += kThreads) c += get(i, &at) == lo && at < end + (1 << bit);
            if (block_sum(c, scratch) < room) end += 1 << bit;
        }
        if (tid == 0) found = 0;
        __syncthreads();
        for (int i = tid; i < total; i += kThreads) {
            const unsigned long long k = get(i, &at);
            if (k > lo || (k == lo && k != 0 && at <= end)) {
                const int j = atomicAdd(&found, 1);
                cand[j] = k, where[j] = at;
            }
        }
        __syncthreads();
        n = found;
    }
    const long out = static_cast<long>(b) * K;
    for (int i = tid; i < n; i += kThreads) {
        const unsigned long long mine = cand[i];
        const int spot = where[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += cand[j] > mine || (cand[j] == mine && where[j] < spot);
        if (rank >= K) continue;
        const int w = spot / V, v = spot - w * V;
        p.out_scores[out + rank] = static_cast<float>(value_of(mine));
        p.parents[out + rank] = b * W + w;
        p.tokens[out + rank] = v;
        p.out_finished[out + rank] =
            v == p.end_token || (p.finished != nullptr && p.finished[b * W + w] != 0);
    }
    for (int i = n + tid; i < K; i += kThreads) {
        p.out_scores[out + i] = -INFINITY;
        p.parents[out + i] = p.tokens[out + i] = -1;
        p.out_finished[out + i] = 1;
    }
}

template <int TYPE, int VEC>
cudaError_t launch_piece(const BeamParams &p, cudaStream_t stream) {
    return launch_overlapped(fa_beam_piece_kernel<TYPE, VEC>, dim3(p.chunks * p.B * p.W), kThreads, 0, stream,
                             p);
}

}  // namespace

cudaError_t launch_beam_select(const BeamParams &p, int type, cudaStream_t stream) {
    const long bits = static_cast<long>(reinterpret_cast<uintptr_t>(p.logits)) /
                          (type == kBeamF32 ? 4 : 2) | p.stride_b | p.stride_w;
    const long align = bits & -bits & 15;  // logits that every row's start is a multiple of
    const int vec = align == 0 || align >= (type == kBeamF32 ? 4 : 8) ? (type == kBeamF32 ? 4 : 8)
                                                                     : static_cast<int>(align);
    cudaError_t e;
    if (type == kBeamF32) {
        e = vec == 4 ? launch_piece<kBeamF32, 4>(p, stream) : vec == 2 ? launch_piece<kBeamF32, 2>(p, stream)
                                                                       : launch_piece<kBeamF32, 1>(p, stream);
    } else if (type == kBeamBF16) {
        e = vec == 8   ? launch_piece<kBeamBF16, 8>(p, stream)
            : vec == 4 ? launch_piece<kBeamBF16, 4>(p, stream)
            : vec == 2 ? launch_piece<kBeamBF16, 2>(p, stream)
                       : launch_piece<kBeamBF16, 1>(p, stream);
    } else {
        e = vec == 8   ? launch_piece<kBeamF16, 8>(p, stream)
            : vec == 4 ? launch_piece<kBeamF16, 4>(p, stream)
            : vec == 2 ? launch_piece<kBeamF16, 2>(p, stream)
                       : launch_piece<kBeamF16, 1>(p, stream);
    }
    if (e != cudaSuccess) return e;
    return launch_overlapped(fa_beam_join_kernel, dim3(p.B), kThreads,
                            (sizeof(double) + sizeof(float)) * p.W, stream, p);
}

}  // namespace fa
