/*
 * fa.h - C ABI of the GB300 (sm_103a) fused exact-attention library, libfa.so.
 *
 * Computes O = softmax(scale * Q K^T [+ causal or 128x128 block mask]) V without writing the
 * N x N score or probability matrices to memory, plus its gradient.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  Layout    Q, K, V, O, dO, dQ, dK, dV are dense, contiguous [B, H, N, d] tensors of one
 *            16-bit type (FA_FP16 or FA_BF16) in device memory; row (b, h, n) starts at element
 *            ((b * H + h) * N + n) * d.  LSE and the backward scratch D are fp32 [B, H, N].
 *            Every device pointer must be 16-byte aligned.
 *  Sizes     d is 64 or 128 (anything else: FA_ERR_UNSUPPORTED).  N >= 1 (ragged N is fine),
 *            B >= 1, H >= 1, B * H * N < 2^31.  scale must be finite and > 0.
 *  Masks     causal != 0: query i sees keys j <= i (queries and keys share one index).
 *            block_mask: device uint8 [T][T] row-major with T = ceil(N / 128), shared by every
 *            (b, h); entry (i, j) != 0 keeps the 128 x 128 score block of query rows
 *            [128 i, 128 i + 128) and key rows [128 j, 128 j + 128).  With both, a score is kept
 *            only if both keep it.  A query row whose every key is masked gets O = 0,
 *            LSE = -inf and zero gradients.  With a block mask T may not exceed 46340
 *            (N <= 5931520; T x T stays below 2^31), else FA_ERR_INVALID.
 *  Ownership The caller owns every buffer.  The library allocates no device memory on any
 *            call; it keeps one device status word per device, created on first use.
 *  Streams   Every call only enqueues work on `stream` (a cudaStream_t; NULL = legacy default
 *            stream) and returns.  The return code covers argument validation and launch
 *            errors only.  Device-side failures (a pipeline wait that ran out of time) are
 *            recorded in the status word and reported by fa_sync_status().
 *  Errors    0 on success, a negative FA_ERR_* code otherwise; nothing is launched when
 *            validation fails.  fa_status_string() names a code.
 *
 * The operation is the one defined by the pages this library follows:
 *  - "FlashAttention-2: better parallelism and work partitioning" (reading notes,
 *    zhongzhuzhou.org): standard attention eq. (2)-(4); forward Algorithm 1 with delayed
 *    normalisation eq. (10)-(11) and the logsumexp eq. (15); backward Algorithm 2 with
 *    P = exp(S - L) eq. (16) and the softmax Jacobian eq. (17); causal masking section.
 *  - FlashAttention post (bluuewhale.github.io): the 1/sqrt(d) scale ("How Attention Is
 *    Computed") and block-sparse FlashAttention ("Block-Sparse FlashAttention").
 *  - The same reading notes, section on MQA/GQA support, for the *_gqa entry points.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FA_FP16 = 0, FA_BF16 = 1, FA_FP32 = 2 /* fa_beam_select's logits only */ } fa_dtype;

enum {
    FA_OK = 0,
    FA_ERR_INVALID = -1,      /* null or misaligned pointer, bad size, bad scale */
    FA_ERR_UNSUPPORTED = -2,  /* head dimension other than 64/128, or no sm_103 device */
    FA_ERR_CUDA = -3,         /* a CUDA runtime call failed (launch, attribute, symbol) */
    FA_ERR_TIMEOUT = -4,      /* a device pipeline wait ran out of time (from fa_sync_status) */
    FA_ERR_INTERNAL = -5,     /* a kernel found its shared memory misplaced (its base not
                                 1024-byte aligned) and returned without computing; never
                                 expected (from fa_sync_status) */
    FA_ERR_FULL = -7,         /* fa_paged_reserve found too few free pages (from fa_sync_status) */
    FA_ERR_INDEX = -6         /* an index array on the device (page ids, token offsets, lengths)
                                 holds a value out of range; what it named was not accessed
                                 (from fa_sync_status), or fa_paged_check found it on the host */
};

/* How fa_rope_frequencies stretches the positions for contexts longer than the trained one. */
enum {
    FA_ROPE_PLAIN = 0,        /* not at all */
    FA_ROPE_LINEAR = 1,       /* every frequency divided by factor */
    FA_ROPE_NTK = 2,          /* base multiplied by factor^(rot_dim / (rot_dim - 2)) */
    FA_ROPE_BY_PARTS = 3,     /* a linear ramp over the pairs between the one that turns `high`
                                 times over original_len (kept) and the one that turns `low`
                                 times (divided by factor); mscale = 0.1 ln(factor) + 1 */
    FA_ROPE_BANDS = 4         /* pairs that turn at least `high` times over original_len kept,
                                 those that turn at most `low` times divided by factor, a linear
                                 blend in the number of turns between */
};

/*
 * Forward.  FlashAttention-2 reading notes, Algorithm 1 (forward) and eq. (15).
 *   q, k, v : [B,H,N,d] inputs (device).
 *   o       : [B,H,N,d] output (device), same dtype.
 *   lse     : [B,H,N] fp32 output (device): LSE_i = m_i + ln(l_i) of the scaled scores.
 *   scale   : multiplies Q K^T before the softmax (1/sqrt(d) for standard attention).
 */
int fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int N,
           int d, int dtype, float scale, int causal, void *stream);

/*
 * Block-sparse forward.  FlashAttention post, "Block-Sparse FlashAttention": a 128 x 128 score
 * block whose mask entry is zero is skipped entirely (never loaded, never multiplied).
 *   block_mask : device uint8 [ceil(N/128)][ceil(N/128)], must not be NULL.
 * Other arguments as fa_fwd.
 */
int fa_fwd_blocksparse(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                       int H, int N, int d, int dtype, float scale, int causal,
                       const uint8_t *block_mask, void *stream);

/*
 * Grouped-query forward.  FlashAttention-2 reading notes, MQA/GQA section: K and V have H_kv
 * heads, H_kv divides H, and query head h attends with K/V head h / (H / H_kv) (consecutive
 * query heads share a K/V head; H_kv = 1 is MQA, H_kv = H is fa_fwd).  K/V are read in place,
 * never copied per query head.
 *   q, o       : [B,H,N,d];  k, v : [B,H_kv,N,d];  lse : [B,H,N] fp32.
 *   block_mask : NULL for dense, otherwise as in fa_fwd_blocksparse.
 * H_kv < 1, or H_kv not dividing H: FA_ERR_INVALID.  Other arguments as fa_fwd.
 */
int fa_fwd_gqa(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
               int H_kv, int N, int d, int dtype, float scale, int causal,
               const uint8_t *block_mask, void *stream);

/*
 * Forward on 8-bit float inputs.  The forward of fa_fwd_gqa with Q, K, V given as e4m3 codes
 * (OCP 8-bit float E4M3: bias 7, 3 mantissa bits, largest 448, NaN = 0x7F/0xFF) and one scale
 * per tensor: element x of Q stands for e4m3(x) * descale_q (likewise K, V).  QK^T and PV run
 * as e4m3 tensor-core products (twice the bf16 rate); the softmax is fp32 as in fa_fwd; the
 * probabilities are rounded to e4m3 before PV (their largest values scaled near the top of the
 * e4m3 range), which bounds O's accuracy by e4m3's 3-bit mantissa rather than bf16's 8 bits.
 *   q       : [B,H,N,d] e4m3 codes (device);  k, v : [B,H_kv,N,d] e4m3 codes (device).
 *   o       : [B,H,N,d] bf16 output (device);  lse : [B,H,N] fp32 output, as in fa_fwd.
 *   descale_q, descale_k, descale_v : finite, > 0.
 *   workspace : at least fa_fwd_fp8_workspace_bytes() bytes, 16-byte aligned: V transposed
 *               ([B,H_kv,d,N rounded up to 16]), written by this call.
 *   block_mask : NULL for dense, otherwise as in fa_fwd_blocksparse.
 * d is 64 or 128.  Other arguments and errors as fa_fwd_gqa.
 */
size_t fa_fwd_fp8_workspace_bytes(int B, int H_kv, int N, int d);
int fa_fwd_fp8(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
               int H_kv, int N, int d, float scale, float descale_q, float descale_k,
               float descale_v, int causal, const uint8_t *block_mask, void *workspace,
               size_t workspace_bytes, void *stream);

/* Bytes of device scratch fa_bwd needs: D (fp32 [B,H,N]), rounded up to 256 bytes. */
size_t fa_bwd_workspace_bytes(int B, int H, int N, int d);

/*
 * Backward.  FlashAttention-2 reading notes, Algorithm 2 with the atomic dQ update replaced by
 * a separate dQ pass: D = rowsum(dO o O) (fa_bwd_preprocess), then dK and dV per key tile
 * (fa_bwd_dkdv), then dQ per query tile (fa_bwd_dq).  Deterministic: no atomics.
 *   o, lse     : the forward's outputs for these q, k, v (same scale, causal, mask).
 *   dout       : [B,H,N,d] gradient of the loss with respect to O.
 *   dq, dk, dv : [B,H,N,d] outputs (device), same dtype as q.
 *   workspace  : device scratch of at least fa_bwd_workspace_bytes() bytes, 16-byte aligned;
 *                overwritten, needs no initialisation.
 *   block_mask : NULL for dense, otherwise as in fa_fwd_blocksparse.
 */
int fa_bwd(const void *q, const void *k, const void *v, const void *o, const void *dout,
           const float *lse, void *dq, void *dk, void *dv, void *workspace,
           size_t workspace_bytes, int B, int H, int N, int d, int dtype, float scale,
           int causal, const uint8_t *block_mask, void *stream);

/*
 * Bytes of device scratch fa_bwd_gqa needs: D (fp32 [B,H,N], rounded up to 256 bytes) plus,
 * when the dK/dV pass splits each K/V head's query group over several CTAs (few K/V heads, so
 * that the GPU is still filled), fp32 partial sums of dK and dV: 2 * splits * B*H_kv*N*d floats.
 * Returns 0 for invalid sizes.  Depends only on the arguments (and fa_debug_set_dkdv_splits).
 */
size_t fa_bwd_gqa_workspace_bytes(int B, int H, int H_kv, int N, int d);

/*
 * Grouped-query backward.  FlashAttention-2 reading notes, MQA/GQA section: the gradient of a
 * shared K/V head is the sum of its query heads' gradients.  The dK/dV pass walks all query
 * heads of a group through one accumulator in tensor memory (and, when split, adds the fp32
 * partials in a fixed order), so the result is deterministic.
 *   q, o, dout, dq : [B,H,N,d];  k, v, dk, dv : [B,H_kv,N,d];  lse : [B,H,N] fp32.
 *   workspace      : at least fa_bwd_gqa_workspace_bytes() bytes, 16-byte aligned.
 * Other arguments as fa_bwd; fa_bwd is this call with H_kv = H.
 */
int fa_bwd_gqa(const void *q, const void *k, const void *v, const void *o, const void *dout,
               const float *lse, void *dq, void *dk, void *dv, void *workspace,
               size_t workspace_bytes, int B, int H, int H_kv, int N, int d, int dtype,
               float scale, int causal, const uint8_t *block_mask, void *stream);

/*
 * Dropout on the attention probabilities (FlashAttention paper detail: dropout is one of the
 * operations fused into the kernel, O = dropout(softmax(S)) V; the pages give no generator).
 * Score (q, k) of query head b*H + h is dropped with probability t / 256, t = the nearest
 * integer to 256 * p_drop (ties to even), and a kept probability is scaled by 256 / (256 - t).
 * The decision is byte (k mod 16) of Philox4x32-10 (Salmon et al., SC 2011) with counter
 * (k div 16, q, b*H + h, offset) and key (seed mod 2^32, seed div 2^32), kept when that byte is
 * >= t; the backward regenerates the same decisions from the same arguments, so nothing is
 * stored.  offset must be below 2^32 (otherwise FA_ERR_INVALID).
 * fa_fwd_dropout: as fa_fwd_gqa; LSE is that of the scores (dropout does not change it).
 * fa_bwd_dropout: as fa_bwd_gqa (same workspace) for the forward with these dropout arguments.
 *   p_drop : 0 <= p_drop < 1 with t <= 255 (otherwise FA_ERR_INVALID); t = 0 is no dropout.
 */
int fa_fwd_dropout(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                   int H, int H_kv, int N, int d, int dtype, float scale, int causal,
                   const uint8_t *block_mask, float p_drop, unsigned long long seed,
                   unsigned long long offset, void *stream);
int fa_bwd_dropout(const void *q, const void *k, const void *v, const void *o, const void *dout,
                   const float *lse, void *dq, void *dk, void *dv, void *workspace,
                   size_t workspace_bytes, int B, int H, int H_kv, int N, int d, int dtype,
                   float scale, int causal, const uint8_t *block_mask, float p_drop,
                   unsigned long long seed, unsigned long long offset, void *stream);

/*
 * The three stages of fa_bwd, exposed so a caller (or a profiler) can order or time them.
 * fa_bwd_preprocess: delta[b,h,i] = sum_k dout[b,h,i,k] * o[b,h,i,k] in fp32 (FlashAttention-2
 *   reading notes, Algorithm 2, precomputation; FlashAttention paper detail, "Technique 2").
 * fa_bwd_dkdv: dK, dV for every key tile from q, k, v, dout, lse and delta.
 * fa_bwd_dq:   dQ for every query tile from q, k, v, dout, lse and delta.
 */
int fa_bwd_preprocess(const void *o, const void *dout, float *delta, int B, int H, int N, int d,
                      int dtype, void *stream);
int fa_bwd_dkdv(const void *q, const void *k, const void *v, const void *dout, const float *lse,
                const float *delta, void *dk, void *dv, int B, int H, int N, int d, int dtype,
                float scale, int causal, const uint8_t *block_mask, void *stream);
int fa_bwd_dq(const void *q, const void *k, const void *v, const void *dout, const float *lse,
              const float *delta, void *dq, int B, int H, int N, int d, int dtype, float scale,
              int causal, const uint8_t *block_mask, void *stream);

/*
 * Backward that allocates nothing: the same computation, arguments and results as fa_bwd,
 * without the workspace.  The pages have no counterpart; this entry point serves callers that
 * cannot allocate device memory themselves, such as a plug-in that a host application hands
 * only its input and output buffers while the application owns every device allocation, or
 * code on a latency-critical path where cudaMalloc's implicit device-wide synchronisation is
 * not acceptable.
 *
 * The D scratch lives in a fixed array compiled into libfa.so: FA_NOALLOC_MAX_ROWS floats
 * (4 MiB) that every GPU which loads the library keeps until the process exits.
 *  - Returns FA_ERR_INVALID, launching nothing, when B * H * N > FA_NOALLOC_MAX_ROWS, or
 *    when the block mask is wider than fa_bwd allows.
 *  - The first call on a device looks up the array's device address with that device current;
 *    make that first call before any stream capture.
 *  - Every call on a device uses the same array, which keeps the last call's values.  Calls
 *    that overlap on the GPU (other streams, other host threads) race on it and corrupt each
 *    other's gradients: order them.  Nothing in it has to start at zero, since each call
 *    writes every value it later reads.
 *  - Neither the call nor its set-up calls cudaMalloc, cudaFree or any allocating routine.
 */
#define FA_NOALLOC_MAX_ROWS (1u << 20)
int fa_bwd_noalloc(const void *q, const void *k, const void *v, const void *o, const void *dout,
                   const float *lse, void *dq, void *dk, void *dv, int B, int H, int N, int d,
                   int dtype, float scale, int causal, const uint8_t *block_mask, void *stream);

/*
 * Decode: a few new query rows per sequence against a KV cache.  FlashAttention-2 reading
 * notes, section on the KV cache (a 1 x d query per generated token against the N cached keys);
 * key ranges of the cache are processed by separate CTAs and merged with the statistic merge of
 * the FlashAttention paper detail, Technique 1.  The kernel is bound by reading K and V.
 *   q, o    : [B,H,Nq,d] (device), Nq >= 1 new rows per sequence;  lse : [B,H,Nq] fp32.
 *   k, v    : [B,H_kv,Nk,d] cache (device), Nk = its capacity; H_kv divides H and query head h
 *             reads K/V head h / (H / H_kv) (as fa_fwd_gqa).
 *   kv_len  : device int32 [B], the number of valid cached positions of each sequence (values
 *             are clamped to [0, Nk]), or NULL for Nk everywhere.
 *   causal  : 0: every new row sees all kv_len[b] keys.  != 0: the new rows are the last Nq
 *             positions of the sequence, row r is position kv_len[b] - Nq + r and sees keys
 *             j <= that position.  A row that sees no key gets O = 0 and LSE = -inf.
 *   workspace, workspace_bytes : device scratch of fa_decode_workspace_bytes() bytes,
 *             16-byte aligned (may be NULL when that is 0): the per-range partial results.
 * Errors as fa_fwd; B*H*Nq and B*H_kv*Nk must be below 2^31.
 */
size_t fa_decode_workspace_bytes(int B, int H, int H_kv, int Nq, int Nk, int d);
int fa_decode(const void *q, const void *k, const void *v, void *o, float *lse,
              const int *kv_len, int B, int H, int H_kv, int Nq, int Nk, int d, int dtype,
              float scale, int causal, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Rotary positions.  Pair j of a row at position p is turned by the angle p * f_j and scaled:
 * (a, c) -> mscale * (a cos - c sin, c cos + a sin).  The first rot_dim elements of a row hold
 * rot_dim / 2 pairs: elements (j, j + rot_dim / 2), or (2j, 2j + 1) when interleaved != 0; the
 * elements behind them are copied as they are.
 *   freq      : device uint64 [rot_dim / 2], 16-byte aligned: f_j as turns per position in units
 *               of 2^-64 turns (rounded down), so that p * f_j modulo a turn is exact integer
 *               arithmetic at any int32 position, negative ones included.
 *   positions : device int32 [B, N], or NULL for 0 .. N - 1 in every sequence.
 *   q, q_out  : [B,H,N,d];  k, k_out : [B,H_kv,N,d], or NULL with H_kv = 0 (Q alone).  H_kv need
 *               not divide H here.
 *   strides   : host array of 12 strides in elements: batch, head and row of q, of q_out, of k and
 *               of k_out (the last six are not read without k); NULL for dense tensors.  Rows are
 *               contiguous; strides are multiples of 8 below 2^39, at least 0 for the inputs and
 *               at least 8 for the outputs (that of an axis of
 *               extent 1 is not looked at), and no two elements of an output may share a place.
 *               An output may be its input with the same strides (in place); any other overlap is
 *               undefined.
 *   inverse   : != 0 turns by -p f_j: with the same mscale this is the transpose of the forward,
 *               which takes the gradients of q_out and k_out to those of q and k.
 * d is 64 or 128; rot_dim is a multiple of 16, at most d (otherwise FA_ERR_UNSUPPORTED); mscale is
 * finite and > 0.  Products and sums are fp32, rounded once; sines and cosines are off by less than
 * 2^-20 in absolute terms, sines of angles below 1/4 by less than 2^-21 relative plus 2^-29.
 *
 * fa_rope_frequencies fills freq (HOST memory, rot_dim / 2 values; rot_dim >= 2 and even) from
 * f_j = base^(-2 j / rot_dim) radians per position, stretched as `scaling` (FA_ROPE_*) says, and
 * *mscale (may be NULL).  factor >= 1, original_len > 0 and 0 < low < high are looked at only
 * where the scaling uses them.
 */
int fa_rope_frequencies(uint64_t *freq, float *mscale, int rot_dim, double base, int scaling,
                        double factor, double original_len, double low, double high);
int fa_rope(const void *q, void *q_out, const void *k, void *k_out, const long long *strides,
            const uint64_t *freq, const int *positions, int B, int H, int H_kv, int N, int d,
            int rot_dim, int dtype, int interleaved, int inverse, float mscale, void *stream);

/*
 * Paged K/V cache.  The cache is a pool of num_pages pages; a page holds page_size positions of
 * all H_kv heads.  A batch brings T new tokens of B sequences, token-major: sequence b has the
 * tokens [q_start[b], q_start[b + 1]) and, counting them, kv_len[b] positions; token i of its n
 * new ones stands at position kv_len[b] - n + i (as in fa_decode).
 *   k_pages, v_pages : [num_pages, H_kv, page_size, d] of one 16-bit type (any order of the first
 *               three axes through `strides`).  page_size is a power of two from 8 to 1024
 *               (otherwise FA_ERR_UNSUPPORTED).
 *   block_table : device int32 [B, max_pages]: page block_table[b][i] holds positions
 *               [i * page_size, (i + 1) * page_size) of sequence b.  Entries behind the last
 *               position are not read.  Sequences may share pages that they only read.
 *   kv_len    : device int32 [B], at most max_pages * page_size.
 *   q_start   : device int32 [B + 1], not decreasing, or NULL: T / B tokens each (B divides T).
 *               Tokens before q_start[0] and from q_start[B] on belong to no sequence (a padded
 *               batch): nothing is written or computed for them, and what their rows hold has no
 *               influence; like all T rows they have to be readable.
 * The index arrays live on the device, so the call cannot refuse a bad value: lengths and offsets
 * are clamped (nothing is appended to such a sequence), a page id outside [0, num_pages) is not
 * accessed (a new token's row is not written, its keys and values read as zeros), and
 * fa_sync_status() returns FA_ERR_INDEX.
 * T (H + 2 H_kv) and num_pages page_size are below 2^31, max_pages page_size at most 2^31 - 1024.
 *
 * fa_paged_check applies the same rules on the host to HOST copies of the arrays, for a scheduler
 * that builds them there: FA_OK, or FA_ERR_INDEX.
 */
int fa_paged_check(const int *block_table, const int *kv_len, const int *q_start, int T, int B,
                   int num_pages, int page_size, int max_pages, int max_q);

/*
 * Appends the new tokens to the cache in one launch: K rotated to its position and V as it is go
 * to their rows; Q, when given, is rotated beside them.
 *   q, q_out  : [T,H,d] or NULL (q_out may be q with the same strides);  k, v : [T,H_kv,d].
 *   strides   : host array of 14 strides in elements: token and head of q, q_out, k and v, then page,
 *               head and row of k_pages and v_pages; NULL for dense tensors; limits as in fa_rope.
 *   freq      : as in fa_rope, or NULL for no rotation (rot_dim, mscale and positions unused).
 *   positions : device int32 [T], the positions to rotate to, or NULL for the places in the cache.
 * A token whose position is below 0 (kv_len[b] < n) has no row and is not stored.  Two tokens that
 * name the same row (tables that share a page they both write) leave it undefined.
 */
int fa_paged_append(const void *q, void *q_out, const void *k, const void *v, void *k_pages,
                    void *v_pages, const long long *strides, const int *block_table,
                    const int *kv_len, const int *q_start, const int *positions,
                    const uint64_t *freq, int T, int B, int H, int H_kv, int d, int num_pages,
                    int page_size, int max_pages, int rot_dim, int dtype, int interleaved,
                    float mscale, void *stream);

/*
 * Attention of every sequence's new tokens (one, a few, or a prompt chunk, mixed in one batch) over
 * its paged cache, which already holds them.  Heads are grouped as in fa_fwd_gqa, at most 128
 * query heads to a K/V head (otherwise FA_ERR_UNSUPPORTED).
 *   q, o      : [T,H,d];  lse : [T,H] fp32 (natural log, as everywhere).
 *   strides   : host array of 10 strides in elements: token and head of q and o, then page, head
 *               and row of k_pages and v_pages; NULL for dense tensors; limits as for the outputs
 *               in fa_rope.  k_pages and v_pages order heads and rows the same way.
 *   max_q     : no sequence brings more new tokens than this (T is always safe, the true maximum is
 *               faster); of a sequence that does, the tokens beyond the first max_q are left out
 *               (their rows of o and lse stay as they were) and FA_ERR_INDEX is reported; the first
 *               max_q see the keys that they see without the bound.
 *   causal    : != 0: row i of sequence b sees keys j <= kv_len[b] - n + i; 0: all kv_len[b] keys.
 *               A row that sees no key gets O = 0 and LSE = -inf.  Whatever the cache holds behind
 *               kv_len[b] (NaN included) has no influence.  Inside it, keys that a row does not see
 *               have none either, but a value there that is not finite may make O of that row (if
 *               it sees any key) NaN: its probability is a zero that may still be multiplied with it.
 * Scores, statistics and sums are fp32; the probabilities are rounded to the inputs' 16-bit type
 * before they are multiplied with V, as in the other attention calls, and O once at the end.
 *   workspace, workspace_bytes : device scratch of fa_paged_attn_workspace_bytes() bytes, 16-byte
 *               aligned (may be NULL when that is 0); it needs no initialisation and keeps nothing
 *               from call to call, but calls that may overlap on the GPU need one each.
 */
size_t fa_paged_attn_workspace_bytes(int T, int B, int H, int H_kv, int d, int max_q,
                                     int page_size, int max_pages);
int fa_paged_attn(const void *q, const void *k_pages, const void *v_pages, void *o, float *lse,
                  const long long *strides, const int *block_table, const int *kv_len,
                  const int *q_start, int T, int B, int H, int H_kv, int d, int num_pages,
                  int page_size, int max_pages, int max_q, int dtype, float scale, int causal,
                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * Keeping a paged cache's tables.  Everything below happens on the device, in the order of the stream:
 * a serving step that branches, grows and drops sequences reads nothing back, and can be captured.
 *   block_table : device int32 [B, max_pages] as above, written by these calls.  An entry is a page id,
 *               or -1 for none; a table starts out as -1 everywhere.  Every entry of a row counts,
 *               those behind the sequence's length too (pages reserved ahead).
 *   refs      : device int32 [num_pages], 16-byte aligned: how many entries hold each page, plus whatever
 *               the caller adds for holds of its own (a prefix to be kept).  A page is free where refs
 *               is 0; refs starts out as zeros.
 * These two are the whole state; the calls leave them consistent, give pages out lowest id first, and
 * so always come to the same tables.  At most 16384 sequences (otherwise FA_ERR_UNSUPPORTED); calls on
 * one table or one refs array have to be ordered by the caller.  Values out of range are not
 * followed and reported as FA_ERR_INDEX by fa_sync_status(), as is a count that would fall below
 * zero (it is left at zero) or an entry to be moved whose page is free.
 *
 * fa_paged_reserve: after it, every page that the batch's new tokens (kv_len, q_start, T as in
 * fa_paged_append) will be written to is held by their sequence alone.  In order of sequence and
 * position: a place without a page gets a free one; a place whose page others hold too gets a free one in
 * its stead, unless all its holders are places of this call: then the first of them keeps the page.
 *   copies    : device int32 [3, B], or NULL: row 0 names the page to copy from, row 1 the one to copy to
 *               and row 2 the rows to copy, for every sequence whose first new token goes behind tokens
 *               on a page that it shared (-1, -1, 0 for the others): arguments for fa_paged_copy.
 *   Sequences with a length or offset out of range get nothing, and none does where offsets decrease.
 *   A page that more of the places hold than refs counts is reported (FA_ERR_INDEX) and kept by the first of them,
 *   also where refs has it as free.
 *   Where the free pages run out, the places that are left get -1 (FA_ERR_FULL from fa_sync_status): a shared
 *   page's hold is given back, nobody else's pages are touched, and appending there is refused as usual.
 *   workspace : at least fa_paged_reserve_workspace_bytes() bytes, 16-byte aligned, as in fa_paged_attn (may be
 *               NULL when that is 0).
 *
 * fa_paged_fork: row b becomes what row parents[b] was; both hold its pages from then on.
 *   parents   : device int32 [B]: -1 leaves row b empty, parents[b] = b as it is; any row may have many
 *               children or none (its pages are given back).
 *   kv_len    : device int32 [B], permuted likewise (0 for an empty row), or NULL.
 *   Entries out of range are handed on as they are; rows that stay as they are and have no other child are not
 *   looked at.
 *
 * fa_paged_free: sequence b keeps the pages of its first keep_len[b] positions (device int32 [B]; 0: a
 * sequence that ends, less than its length: drafted tokens that were refused) and gives the others back.
 *
 * fa_paged_compact: moves the live pages to the front of the pool: with n of them, the k-th of those with
 * ids from n on takes the place of the k-th free page before n.  Table and refs follow; the data has to be
 * moved by fa_paged_copy with the lists that it leaves:
 *   src, dst  : device int32 [num_pages / 2] (at least one), of which the first *count are written (the others stay).
 *   count     : device int32, how many pages move.
 * fa_paged_compact and fa_paged_fork need no page size: max_pages is below 2^28.
 *
 * fa_paged_copy: the first rows[i] rows (rows NULL: all) of page src[i] to page dst[i], of all heads, of K
 * and of V, in all layers, for i < n.
 *   k_pages, v_pages : L layers of pages, as in fa_paged_append; written.
 *   strides   : host array of 8 strides in elements: layer, page, head and row of k_pages and of v_pages;
 *               NULL for dense tensors [L, num_pages, H_kv, page_size, d]; limits as for the outputs in
 *               fa_rope.
 *   src, dst, rows : device int32 [n].  Pairs with a negative page are left out.  A page may be copied to
 *               many; one that is copied to must not occur otherwise.
 *   count     : device int32: no more than that many pairs, or NULL.
 */
size_t fa_paged_reserve_workspace_bytes(int T, int B, int num_pages, int page_size);
int fa_paged_reserve(int *block_table, const int *kv_len, const int *q_start, int *refs, int *copies,
                     int T, int B, int num_pages, int page_size, int max_pages, void *workspace,
                     size_t workspace_bytes, void *stream);
int fa_paged_fork(int *block_table, int *kv_len, const int *parents, int *refs, int B, int num_pages,
                  int max_pages, void *stream);
int fa_paged_free(int *block_table, const int *keep_len, int *refs, int B, int num_pages,
                  int page_size, int max_pages, void *stream);
int fa_paged_compact(int *block_table, int *refs, int *src, int *dst, int *count, int B, int num_pages,
                     int max_pages, void *stream);
int fa_paged_copy(void *k_pages, void *v_pages, const long long *strides, const int *src,
                  const int *dst, const int *rows, const int *count, int n, int L, int H_kv, int d,
                  int num_pages, int page_size, void *stream);

/*
 * Beam search's selection.  Each of B requests has W beams; candidate (w, v) continues beam w with token v
 * and scores scores[b][w] + logits[b][w][v] - ln sum_u e^logits[b][w][u].  The K best candidates of a
 * request are returned, best first, equal ones by the lowest w V + v; scores are compared before they
 * are rounded to fp32.
 *   logits    : device [B, W, V] of FA_FP16, FA_BF16 or FA_FP32 (dtype), aligned to an element.
 *   strides   : host array of 2 strides in elements (request, beam), at least 0 and below 2^39; NULL for a
 *               dense tensor.
 *   scores    : device fp32 [B, W].
 *   finished  : device uint8 [B, W], or NULL.  A beam that has ended (not 0) has one candidate: end_token,
 *               with the beam's score.  Its logits are not read.
 *   end_token : -1 for none (only without finished).
 *   out_scores, parents, tokens, out_finished : device [B, K]; parents (int32) are places in the batch,
 *               b W + w, as fa_paged_fork wants them where K = W; out_finished (uint8) is 1 where the
 *               token is end_token or the parent had ended.  Where K = W, out_scores may be scores and
 *               out_finished finished (in place).
 * Only finite scores are candidates: a token of logit -inf is none, nor is any of a beam whose score or
 * whose logits' sum is not finite (a NaN or +inf among them).  Where a request has fewer than K, the
 * places left have score -inf, parent and token -1 and out_finished 1.
 * W V, B K and B W (V div 4096 + 1) are below 2^31; K is at most 128 and W at most 2048 (otherwise
 * FA_ERR_UNSUPPORTED).  Sums are fp32.
 *   workspace : at least fa_beam_select_workspace_bytes() bytes, 16-byte aligned, as in fa_paged_attn (may be
 *               NULL when that is 0).
 */
size_t fa_beam_select_workspace_bytes(int B, int W, int V, int K);
int fa_beam_select(const void *logits, const long long *strides, const float *scores,
                   const uint8_t *finished, float *out_scores, int *parents, int *tokens,
                   uint8_t *out_finished, int B, int W, int V, int K, int dtype, int end_token,
                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Synchronises `stream`, then returns and clears the current device's status word:
 * FA_OK, FA_ERR_TIMEOUT (a kernel gave up on a pipeline wait and returned early; its outputs
 * are undefined), FA_ERR_INTERNAL (a kernel refused to run on a misaligned shared-memory base;
 * its outputs are undefined), FA_ERR_INDEX (a paged call met an index out of range), FA_ERR_FULL (a cache
 * ran out of pages; the first of these two that was met is reported, where neither of the other two
 * is) or FA_ERR_CUDA (the stream reported an error).
 */
int fa_sync_status(void *stream);

/* Static string naming a return code. */
const char *fa_status_string(int code);

/*
 * Test and diagnostics hooks (process-wide; they affect launches made after the call).
 * fa_debug_set_visit_log: when buf != NULL, every kernel ORs a bit into
 *   buf[((b*H + h) * T + i) * T + j] for each score tile (query tile i, key tile j) it
 *   computes: bit 0 forward, bit 1 dK/dV, bit 2 dQ.  bytes must cover B*H*T*T of the launches
 *   that follow, rounded up to a multiple of 4 (the bits are set by 32-bit atomic ORs); buf
 *   must be 4-byte aligned (otherwise FA_ERR_INVALID).  NULL (or bytes = 0) turns logging off.
 * fa_debug_set_wait_limit_ns: bound on every device pipeline wait (default 2 s; 0 restores it).
 * fa_debug_set_fault: 0 = none; 1 = the forward's load warp skips the first key tile of each
 *   CTA; 2 = the dK/dV pass's load warp skips its first Q tile; 3 = the dQ pass's load warp
 *   skips its first K tile; 4 = paged attention's K load warp skips the first key tile of each
 *   CTA.  The bounded waits then run out, the kernel returns early and
 *   fa_sync_status() reports FA_ERR_TIMEOUT; other values: FA_ERR_INVALID.
 * fa_debug_set_dkdv_splits: 0 = automatic; s > 0 splits every K/V head's query group of
 *   fa_bwd_gqa over min(s, H / H_kv) dK/dV CTAs per key tile (changes the workspace size).
 *   Negative: FA_ERR_INVALID.
 * fa_debug_paged_pieces: how fa_paged_attn would spread a batch's work over up to `ctas` CTAs, worked
 *   out on the host from HOST copies of kv_len and q_start, with units of up to `tiles` (1 or 2)
 *   query tiles of tile_toks tokens: 9 ints per piece, in order (CTA, sequence, K/V head, first
 *   token, tokens, first and end key tile, key tiles of the unit, the CTA that holds its last
 *   piece).  Returns the number of pieces (only the first max_pieces are stored) or an error.
 */
int fa_debug_paged_pieces(const int *kv_len, const int *q_start, int T, int B, int H_kv,
                          int page_size, int max_pages, int max_q, int tile_toks, int tiles,
                          int causal, int ctas, int *pieces, int max_pieces);
int fa_debug_set_visit_log(uint8_t *buf, size_t bytes);
int fa_debug_set_wait_limit_ns(unsigned long long ns);
int fa_debug_set_fault(int mode);
int fa_debug_set_dkdv_splits(int splits);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
