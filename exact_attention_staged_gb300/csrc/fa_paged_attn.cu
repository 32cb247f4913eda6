// fa_paged_attn.cu - attention of the new tokens of every sequence over its paged cache.
//
// Row i of the n new tokens of sequence b sees the keys j <= kv_len[b] - n + i (causal) or all
// kv_len[b] of them: O = softmax(scale q K^T) V and the logsumexp, by the online softmax
// (FlashAttention-2 reading notes, Algorithm 1) over the sequence's pages.
//
// One warp per (token, query head): a lane holds D / 32 elements of the row, scores come from a
// shuffle sum, the running maximum and sum are in log2 units.
#include "paged.cuh"

namespace fa {
namespace {

constexpr int kSimpleWarps = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(kSimpleWarps * 32) fa_paged_attn_kernel(const PagedAttnParams p) {
    constexpr int kW = D / 64;  // 32-bit words (element pairs) per lane
    const PagedView &c = p.c;
    const long w = static_cast<long>(blockIdx.x) * kSimpleWarps + warp_id();
    if (w >= static_cast<long>(c.T) * c.H) return;
    const int t = static_cast<int>(w / c.H), h = static_cast<int>(w % c.H);
    const int lane = lane_id();
    const int b = paged_find(c, t);
    if (b < 0) return;
    const PagedSeq s = paged_seq(c, b);
    if (s.bad && lane == 0) paged_report(c);
    const int i = t - s.tok0;
    if (i < 0 || i >= s.n) return;
    const int last = p.causal ? s.len - s.n + i : s.len - 1;
    const int kvh = h / (c.H / c.Hkv);
    auto words = [&](const uint16_t *row, float2 *x) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(row) + lane * kW;
#pragma unroll
        for (int e = 0; e < kW; ++e) x[e] = unpack2<BF16>(src[e]);
    };
    float2 q[kW], acc[kW];
    words(p.q + t * p.q_t + h * p.q_h, q);
#pragma unroll
    for (int e = 0; e < kW; ++e) acc[e] = make_float2(0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    int page = -1;
    for (int j = 0; j <= last; ++j) {
        const int row = j & ((1 << c.page_shift) - 1);
        if (row == 0) {
            page = paged_page(c, b, j);
            if (page < 0 && lane == 0) paged_report(c);
        }
        if (page < 0) continue;
        float2 k[kW], v[kW];
        words(p.k_pages + page * p.kp_p + kvh * p.kp_h + row * p.kp_r, k);
        words(p.v_pages + page * p.vp_p + kvh * p.vp_h + row * p.vp_r, v);
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < kW; ++e) x = fmaf(q[e].x, k[e].x, fmaf(q[e].y, k[e].y, x));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        x *= p.scale_log2;
        const float mn = fmaxf(m, x);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float alpha = exp2f(m - mu), e2 = exp2f(x - mu);
        m = mn;
        l = l * alpha + e2;
#pragma unroll
        for (int e = 0; e < kW; ++e) {
            acc[e].x = fmaf(e2, v[e].x, acc[e].x * alpha);
            acc[e].y = fmaf(e2, v[e].y, acc[e].y * alpha);
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.o + t * p.o_t + h * p.o_h) + lane * kW;
#pragma unroll
    for (int e = 0; e < kW; ++e) dst[e] = pack2<BF16>(acc[e].x * inv, acc[e].y * inv);
    if (lane == 0)
        p.lse[static_cast<long>(t) * c.H + h] =
            l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

template <int D, bool BF16>
cudaError_t launch_attn_t(const PagedAttnParams &p, cudaStream_t stream) {
    const long warps = static_cast<long>(p.c.T) * p.c.H;
    fa_paged_attn_kernel<D, BF16><<<static_cast<unsigned>((warps + kSimpleWarps - 1) / kSimpleWarps),
                                    kSimpleWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnParams &p, int d, bool bf16, cudaStream_t stream) {
    if (d == 64) return bf16 ? launch_attn_t<64, true>(p, stream)
                             : launch_attn_t<64, false>(p, stream);
    return bf16 ? launch_attn_t<128, true>(p, stream) : launch_attn_t<128, false>(p, stream);
}

}  // namespace fa
