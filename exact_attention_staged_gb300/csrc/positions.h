// positions.h - parameter blocks and launchers of the rotary-position and paged-cache kernels.
#pragma once

#include "fa_internal.h"

namespace fa {

// Rotary positions (see fa_rope.cu).  Strides in elements.
struct RopeSide {
    const uint16_t *in;       // [B, heads, N, d], elements of a row contiguous
    uint16_t *out;            // may be `in`
    long in_b, in_h, in_n, out_b, out_h, out_n;
};
struct RopeParams {
    RopeSide q, k;            // k unused with Hkv == 0
    const unsigned long long *freq;  // [rot / 2] turns per position, in units of 2^-64
    const int *positions;     // [B, N], or nullptr for 0 .. N - 1
    long rows;                // B * N
    int N, H, Hkv;
    int rot;                  // rotated elements of a row, a multiple of 16
    int chunk;                // heads per thread (set by the launcher)
    int inverse;              // 1: the transpose
    float mscale;
};

// The paged cache as its readers and writers see it (see fa_paged.cu).  Page `id` of the cache
// holds positions [i * page_size, (i + 1) * page_size) of the sequence whose table has it at i.
struct PagedView {
    const int *table;         // [B, max_pages] page ids
    const int *kv_len;        // [B] cached positions of each sequence, the new tokens included
    const int *q_start;       // [B + 1] first token of each sequence, or nullptr: T / B each
    int T, B, H, Hkv;
    int num_pages, page_shift, max_pages;  // page_size = 1 << page_shift
    int max_q;                // no sequence has more new tokens
    int *status;              // device status word
};

struct PagedAppendParams {
    PagedView c;
    const uint16_t *q, *k, *v;       // [T, heads, d]; q may be nullptr
    uint16_t *q_out, *k_pages, *v_pages;
    long q_t, q_h, qo_t, qo_h, k_t, k_h, v_t, v_h;   // token and head strides, elements
    long kp_p, kp_h, kp_r, vp_p, vp_h, vp_r;         // page, head and row strides
    const unsigned long long *freq;  // nullptr: no rotation
    const int *positions;            // [T] for the rotation, or nullptr: the places in the cache
    int rot;
    int chunks;                      // warps per token (set by the launcher)
    unsigned blocks;                 // that move data (set by the launcher)
    float mscale;
};

struct PagedAttnParams {
    PagedView c;
    uint16_t *o;
    float *lse;                      // [T, H]
    long o_t, o_h;                   // token and head strides, elements
    int rep;                         // query heads per K/V head
    int tile_toks;                   // tokens per query tile: floor(128 / rep)
    int q_box_toks;                  // tokens per Q box of the tensor map
    int q_bufs;                      // Q buffers where a unit has one query tile: 2 up to 64 rows
    int part_rows;                   // rows of a partial result's slot
    float scale_log2;                // scale * log2(e)
    int causal;
    int device;                      // host only: the current device
    // a unit that a border cuts: CTA c's piece that starts inside a unit goes to slot 2c, its piece
    // that starts one but does not end it to slot 2c + 1, and cut[c] says what to merge
    float4 *part_o;                  // [slots][d / 4][part_rows] unnormalised, 4 columns each
    float2 *part_ml;                 // [slots][part_rows] running max (log2) and sum
    int4 *cut;                       // [2 * CTAs], or nullptr: no unit has more than one key tile
    Ctl ctl;
};

struct PagedMaps {
    CUtensorMap q;                   // (d, rep, H_kv, T), boxes 64 x rep x 1 x q_box_toks
    CUtensorMap k, v;                // (d, rows, H_kv, pages) or (d, H_kv, rows, pages) by stride,
                                     // boxes of 64 elements of min(page_size, 128) rows
    int rows_inner;                  // 1: the first of these orders
};

constexpr int kPagedCtas = 152;      // one per SM

constexpr int kErrIndex = -6;  // an index array on the device holds a value out of range

// A launch that may overlap the end of the grid before it in the stream (programmatic stream
// serialization): the kernel calls griddep_wait() before it touches global memory, so only its
// launch and set-up are early, and griddep_launch_dependents() lets its own successor do the same.
template <class... KernelArgs, class... Args>
cudaError_t launch_overlapped(void (*kernel)(KernelArgs...), dim3 grid, unsigned threads, size_t smem,
                              cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_rope(const RopeParams &p, int d, bool bf16, bool inter, cudaStream_t stream);
cudaError_t launch_paged_append(const PagedAppendParams &p, int d, bool bf16, bool inter,
                                cudaStream_t stream);
// Clusters of `ctas` CTAs, one for each of up to `units` units; ctas 0: one line of units over all SMs.
struct PagedClusters {
    int ctas;
    long units;
};
// tiles: query tiles per unit, 1 or 2
cudaError_t launch_paged_attn(const PagedMaps &m, const PagedAttnParams &p, int d, bool bf16,
                              int tiles, PagedClusters cl, cudaStream_t stream);

}  // namespace fa
