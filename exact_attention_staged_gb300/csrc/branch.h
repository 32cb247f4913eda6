// branch.h - parameter blocks and launchers of decoding with branches: the page tables' upkeep
// (fa_pages.cu) and beam selection (fa_beam.cu).
#pragma once

#include "positions.h"

namespace fa {

constexpr int kErrFull = -7;  // too few free pages

// A page is free where refs is 0; a table's entry is a page id, or below 0 for none.
struct PageTables {
    int *table;               // [B, max_pages]
    int *refs;                // [num_pages] holders of each page
    int B, num_pages, max_pages, page_shift;
    int *status;              // device status word
    int device;               // host only: the current device
};

struct PagedReserveParams {
    PagedView c;              // the batch; c.table is t.table
    PageTables t;
    int *copies;              // [3, B]: page to copy from, page to copy to, rows; or nullptr
    int *fresh;               // workspace, where reserve_shape() has none: the pages given out, in order
};

struct PagedForkParams {
    PageTables t;
    int *kv_len;              // [B] or nullptr
    const int *parents;       // [B]
    int shift;                // 2^shift columns of the table per block (set by the launcher)
};

struct PagedFreeParams {
    PageTables t;
    const int *keep_len;      // [B]
};

struct PagedCompactParams {
    PageTables t;
    int *src, *dst;           // [num_pages / 2]
    int *count;
    int apply;                // table and refs too, in the same launch (set by the launcher)
};

struct PagedCopySide {
    uint16_t *base;
    long layer, page, outer, inner;  // strides in elements
};
struct PagedCopyParams {
    PagedCopySide k, v;
    const int *src, *dst, *rows, *count;
    int n, L, num_pages;
    // a page's runs are its heads, with the rows as inner index, or the other way round
    int heads, page_size, rows_inner;
    int piece_shift;                 // a head's row is 2^piece_shift pieces of 16 bytes
    unsigned parts, per;             // blocks of a pair, and runs of each (set by the launcher)
    int *status;
};

struct BeamParams {
    const void *logits;
    long stride_b, stride_w;         // elements
    const float *scores;             // [B, W]
    const uint8_t *finished;         // [B, W] or nullptr
    float *out_scores;               // [B, K]
    int *parents, *tokens;           // [B, K]
    uint8_t *out_finished;           // [B, K]
    int B, W, V, K, end_token;
    int pieces, piece_len;           // pieces of a row, and their logits (whole tiles)
    int ctas;                        // per request, or 0: a grid over all pieces, and one that joins them
    unsigned long long *keys;        // workspace [B * W][pieces][K]
    float2 *stats;                   // workspace [B * W][pieces]: maximum, sum of e^(x - maximum)
};

cudaError_t launch_paged_reserve(const PagedReserveParams &p, cudaStream_t stream);
cudaError_t launch_paged_fork(PagedForkParams p, cudaStream_t stream);
cudaError_t launch_paged_free(const PagedFreeParams &p, cudaStream_t stream);
cudaError_t launch_paged_compact(PagedCompactParams p, cudaStream_t stream);
cudaError_t launch_paged_copy(PagedCopyParams p, cudaStream_t stream);
struct ReserveShape {
    int threads, ctas;
};
ReserveShape reserve_shape(int T, int B, int num_pages, int page_size);

// Sequences that one call may have: their places are kept in shared memory.
constexpr int kBranchMaxSeqs = 16384;

enum BeamType { kBeamF16 = 0, kBeamBF16 = 1, kBeamF32 = 2 };
constexpr int kBeamThreads = 256;
constexpr int kBeamNoted = 4096;        // maxima that a CTA notes: a piece has as many times its threads in tiles
// Logits per load, 16 bytes or what the rows' starts are aligned to.
inline int beam_vec(const void *logits, long stride_b, long stride_w, int type) {
    const long size = type == kBeamF32 ? 4 : 2, most = 16 / size;
    const long bits = static_cast<long>(reinterpret_cast<uintptr_t>(logits)) / size | stride_b | stride_w;
    const long align = bits & -bits;  // 0: every row starts at address 0, as it were
    return static_cast<int>(align == 0 || align > most ? most : align);
}
// A thread's logits of a tile: twice as many where a load brings several 16-bit ones.
constexpr int beam_elems(int type, int vec) { return type != kBeamF32 && vec >= 4 ? 32 : 16; }
constexpr int kBeamMaxK = 128;
constexpr int kBeamMaxWidth = 2048;     // beams of a request
cudaError_t launch_beam_select(const BeamParams &p, int type, int vec, cudaStream_t stream);

// A launch of `clusters` clusters of `ctas` CTAs that may overlap the end of the grid before it.  `smem` and the
// kernel's static part are 48 KB at most, or allowed by allow_smem() before.
template <class Params>
cudaError_t launch_clusters(void (*kernel)(Params), int clusters, int ctas, int threads, size_t smem,
                            cudaStream_t stream, const Params &p) {
    if (ctas > 8) {  // more than every device has to allow
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace fa
