/*
 * li.h -- C ABI of libli, a B200 (sm_100a) LightningIndexer.
 *
 * The operation (mindspore.ops.lightning_indexer page, ".. math::"; CANN
 * LightningIndexerV2 guide, "三步计算流程"; VllmQuantLightningIndexer README,
 * "功能说明"): for every query token and every key it may see,
 *
 *     s(t) = sum_h W[h] * ReLU( [Scale_Q[h] * Scale_K[t] *] (q_h . k_t) )
 *
 * then the sparse_count keys with the largest s (ties: lower key index first)
 * are returned as int32 indices, optionally with their fp32 scores.
 *
 * Conventions shared by every entry point:
 *   - The caller owns all memory.  Every tensor pointer is a DEVICE pointer to
 *     a contiguous tensor (PA key blocks may be strided, see key_block_stride),
 *     16-byte aligned.  The library allocates nothing and never synchronises
 *     the stream, except li_read_device_status, which says so.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Every launch is asynchronous on it.
 *   - A return value other than LI_OK means that nothing was launched; the
 *     reason is in li_last_error() (a thread-local string).
 *   - Errors that only the device can see (an actual length beyond the tensor
 *     or the declared bound, a block id outside the pool, a negative dequant
 *     scale, a bounded wait that expired) never fault: the kernels clamp or
 *     skip the access and OR a bit into the status word at the start of the
 *     workspace.  Read it with li_read_device_status.
 */
#ifndef LI_H
#define LI_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define LI_API __attribute__((visibility("default")))
#else
#define LI_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LI_OK = 0,
    LI_ERR_NULL = 1,         /* a required pointer is NULL                        */
    LI_ERR_SHAPE = 2,        /* a dimension or attribute is out of range          */
    LI_ERR_DTYPE = 3,        /* dtype combination not allowed                     */
    LI_ERR_LAYOUT = 4,       /* layout combination not allowed                    */
    LI_ERR_UNSUPPORTED = 5,  /* allowed by the pages but not built here           */
    LI_ERR_WORKSPACE = 6,    /* workspace missing, too small or misaligned        */
    LI_ERR_CUDA = 7,         /* a CUDA runtime call failed                        */
    LI_ERR_DEVICE = 8        /* li_read_device_status: the device flagged a problem */
} li_status;

typedef enum { LI_BF16 = 0, LI_FP16 = 1, LI_FP32 = 2, LI_FP8_E4M3 = 3, LI_INT8 = 4 } li_dtype;
typedef enum { LI_BSND = 0, LI_TND = 1, LI_PA_BSND = 2 } li_layout;

/* Bits of the device status word (li_read_device_status). */
#define LI_DEV_BAD_QLEN      0x01  /* query length / prefix sum out of range (clamped)  */
#define LI_DEV_BAD_KLEN      0x02  /* key length / prefix sum out of range (clamped)    */
#define LI_DEV_BAD_BLOCK     0x04  /* block_table entry outside [0, num_blocks) (skipped) */
#define LI_DEV_NEG_SCALE     0x08  /* negative dequant scale (the fold needs scales >= 0) */
#define LI_DEV_TIMEOUT       0x10  /* a bounded pipeline wait expired                   */

/*
 * Op attributes and dimensions (mindspore page, "参数" / "关键字参数"; CANN
 * guide, "约束说明"; README, "参数说明").
 *   layout_q       LI_BSND: query [B,S1,N1,D], weights [B,S1,N1]
 *                  LI_TND : query [T1,N1,D],   weights [T1,N1]
 *   layout_k       LI_BSND: key [B,S2,N2,D]; LI_TND: key [T2,N2,D];
 *                  LI_PA_BSND: key [num_blocks,block_size,N2,D] addressed via block_table.
 *                  Without PA, layout_k must equal layout_q.
 *   dtype_qk       LI_BF16 / LI_FP16 (li_indexer); LI_FP8_E4M3 / LI_INT8 (li_quant_indexer)
 *   dtype_w        LI_BF16 / LI_FP16 / LI_FP32
 *   dtype_scale    LI_FP32 / LI_FP16 (li_quant_indexer only)
 *   N1             query heads, 1..64;  N2 key heads, must be 1
 *   D              head dim: 128, or 64 for 16-bit q/k (the TileLang test shape)
 *   num_blocks, block_size, max_blocks_per_seq
 *                  PA pool geometry; block_size a multiple of 16 in [16, 1024]
 *   key_block_stride  elements between consecutive PA blocks (0 = dense
 *                  block_size*N2*D); lets axis 0 of the pool be non-contiguous
 *   sparse_count   k, 1..8192 (CANN guide, "约束说明")
 *   sparse_mode    0 = every key inside the actual length; 3 = right-down causal:
 *                  key t is visible to query i of batch b iff t <= i + Sk_b - Sq_b
 *   pre_tokens, next_tokens  reserved; must be INT64_MAX
 *   return_value   1 = also write sparse_values (fp32)
 *   max_seqlen_k   host-side upper bound on every actual key length (0 = S2 for
 *                  BSND, T2 for TND, max_blocks_per_seq*block_size for PA).  It
 *                  sizes the workspace; longer actual lengths are clamped and flagged.
 *   init_num, local_num  sink tokens and local window (the MT lightning_indexer
 *                  attributes of the open-sourcing issue): the first init_num and
 *                  the last local_num visible keys of every row are always
 *                  selected, the best other visible keys fill the remaining
 *                  slots, all ordered by score.  0 = off; init_num + local_num
 *                  must not exceed sparse_count.
 *   cmp_ratio      compressed keys (CANN LightningIndexerV2 guide): every key
 *                  stands for cmp_ratio original tokens; 0 or 1 = none; a power
 *                  of two up to 128.  Indices count compressed keys.
 *   cmp_residual_k device int32 [B]: original key tokens left over after the
 *                  last whole compressed key, each < cmp_ratio.  Required when
 *                  cmp_ratio > 1 and sparse_mode == 3 (then a key is visible once
 *                  all of its original tokens are: key t is visible to query i iff
 *                  (t+1)*cmp_ratio - 1 <= i + Sk*cmp_ratio + residual - Sq);
 *                  ignored otherwise.  A residual outside [0, cmp_ratio) is
 *                  clamped and flagged with LI_DEV_BAD_KLEN.
 *   reserved       must be 0
 */
typedef struct {
    int32_t layout_q, layout_k;
    int32_t dtype_qk, dtype_w, dtype_scale;
    int32_t B, S1, S2, T1, T2, N1, N2, D;
    int32_t num_blocks, block_size, max_blocks_per_seq;
    int64_t key_block_stride;
    int32_t sparse_count, sparse_mode;
    int64_t pre_tokens, next_tokens;
    int32_t return_value;
    int32_t max_seqlen_k;
    int32_t init_num, local_num;
    int32_t cmp_ratio;
    int32_t reserved;
    const int32_t *cmp_residual_k;
} li_params;

/*
 * Output shape (CANN guide, "输出 shape 的推导依据"; mindspore page, "返回").
 * BSND query: sparse_indices is [B, S1, N2, k] (ndim 4); TND: [T1, N2, k]
 * (ndim 3).  sparse_values has the same shape when return_value is set.
 * out_dims must hold 4 entries.  Host only; validates params.
 */
LI_API li_status li_output_shape(const li_params *p, int64_t out_dims[4], int32_t *ndim);

/* Bytes of device workspace that li_indexer / li_quant_indexer need for `p`
 * (status word, scheduler tables and one fp32 score row per query).  Host only. */
LI_API li_status li_workspace_size(const li_params *p, size_t *bytes);

/*
 * The indexer on 16-bit query/key (mindspore page, whole signature; CANN guide,
 * "函数原型").
 *   query, key, weights   device tensors in the layouts above
 *   act_seq_q  int32 [B]: per-batch query lengths for BSND (NULL = S1 each), or
 *              prefix sums without a leading 0 for TND (required)
 *   act_seq_k  int32 [B]: per-batch key lengths for BSND (NULL = S2 each) and
 *              PA (required), or prefix sums for TND (required)
 *   block_table int32 [B, max_blocks_per_seq], PA only: physical block of each
 *              logical key block
 *   sparse_indices  int32 [rows, k] output; slots past min(k, visible) are -1
 *   sparse_values   fp32 [rows, k] output (NULL iff return_value == 0); padding -inf
 *   workspace       device buffer of li_workspace_size bytes, 256-byte aligned;
 *                   it must not be shared by calls that may run concurrently
 */
LI_API li_status li_indexer(const li_params *p, const void *query, const void *key, const void *weights,
                     const int32_t *act_seq_q, const int32_t *act_seq_k,
                     const int32_t *block_table, int32_t *sparse_indices, float *sparse_values,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * The quantised indexer (VllmQuantLightningIndexer README, "功能说明" and
 * "参数说明"): q/k are fp8 e4m3 or int8, and the per-token-head dequant
 * scales multiply the dot product before the ReLU.  int8 q/k accumulate
 * exactly in s32 (|q.k| <= 2^21 for D = 128) and are converted to fp32.
 *   q_scale  dtype_scale (fp32 or fp16), same layout as weights ([B,S1,N1] or [T1,N1])
 *   k_scale  dtype_scale per key token: [B,S2,N2], [T2,N2] or [num_blocks,block_size,N2]
 * Scales must be >= 0 (then ReLU(sq*sk*x) = sq*sk*ReLU(x), which the kernel
 * uses); a negative scale is flagged with LI_DEV_NEG_SCALE.  Other arguments
 * as li_indexer.
 */
LI_API li_status li_quant_indexer(const li_params *p, const void *query, const void *key,
                           const void *weights, const void *q_scale, const void *k_scale,
                           const int32_t *act_seq_q, const int32_t *act_seq_k,
                           const int32_t *block_table, int32_t *sparse_indices,
                           float *sparse_values, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * The Top-k stage on its own (CANN guide, "三步计算流程" step 3, with the
 * deterministic ordering of "确定性计算"): for each of `rows` fp32 score rows
 * (row r starts at scores + r*ld and its first row_len[r] entries are the
 * candidates; row_len NULL = ld for every row), write the k largest as
 * (index, value) pairs ordered by value descending, ties by lower index; pad
 * with -1 / -inf.  -0.0 counts as +0.0.  ld must be a multiple of 4.
 * sparse_values may be NULL.  Needs no workspace.
 */
LI_API li_status li_topk(const float *scores, int64_t ld, const int32_t *row_len, int32_t rows,
                  int32_t k, int32_t *sparse_indices, float *sparse_values, void *stream);

/*
 * li_indexer for callers that cannot hand the library any device memory of
 * their own.  The pages have no counterpart to it; it is an addition of this
 * library.
 *
 * Some callers cannot allocate device memory: an operator interface that
 * passes a kernel only its input and output tensors and has no workspace
 * mechanism, or a serving loop that keeps cudaMalloc off its hot path (the
 * call can synchronise the device and fragment a pre-reserved pool).  This
 * entry point takes the same arguments as li_indexer minus the workspace and
 * uses instead a scratch array of LI_NOALLOC_SCRATCH_BYTES compiled into the
 * library: every GPU that loads the library holds that memory until the
 * process exits.  It calls no allocator itself.
 *
 *   - Problems whose li_workspace_size exceeds LI_NOALLOC_SCRATCH_BYTES are
 *     rejected with LI_ERR_WORKSPACE before anything is launched; use
 *     li_indexer with a workspace for them.
 *   - The first call on a device looks up that device's copy of the array
 *     (cudaGetSymbolAddress); make that first call before any stream capture.
 *     The address belongs to the device's current context: a call made after
 *     that context was destroyed and re-created (cudaDeviceReset) looks it up
 *     again, so that call too should come before any capture.
 *   - All calls on a device share the one array and it keeps the contents of
 *     the last call.  Nothing in it has to start at zero (each call's
 *     scheduler overwrites the status and tables, and every score is written
 *     before it is read), but calls that may overlap on the GPU -- concurrent
 *     streams, or threads launching at the same time -- race on it.
 *   - The device status word of these calls sits in the library's scratch
 *     and is not exposed; use li_indexer with a workspace when the LI_DEV_*
 *     bits are needed.
 */
#define LI_NOALLOC_SCRATCH_BYTES (32u << 20)
LI_API li_status li_indexer_noalloc(const li_params *p, const void *query, const void *key,
                                    const void *weights, const int32_t *act_seq_q,
                                    const int32_t *act_seq_k, const int32_t *block_table,
                                    int32_t *sparse_indices, float *sparse_values, void *stream);

/*
 * Sparse attention over the selected keys: the consumer of the indexer's
 * output (CANN TileLang LightningIndexer guide, section "LightningIndexer 在
 * 稀疏注意力中的地位": an explicit index tensor names, for every query token,
 * the key/value subset it attends to, so attention costs O(N*S) instead of
 * O(N^2); the open-sourcing issue, section 3: the forward's sparse_indices feed
 * Sparse FlashAttention).  The pages give no formula of their own for it; this
 * library computes scaled dot-product attention restricted to each row's
 * selected keys, with one key/value head shared by all query heads:
 *
 *     J      = entries j of the row's index list with 0 <= j < Sk_b
 *     out_h  = sum_{j in J} softmax_j(scale * q_h . k_j) * v_j
 *     lse_h  = log sum_{j in J} exp(scale * q_h . k_j)
 *
 * and out = 0, lse = -inf for rows with J empty and for BSND padding rows.
 *
 *   layout_q       LI_BSND: query/out [B,S1,N1,D]; LI_TND: [T1,N1,D]
 *   layout_kv      LI_BSND: key [B,S2,1,D], value [B,S2,1,Dv]; LI_TND: [T2,1,D] /
 *                  [T2,1,Dv]; LI_PA_BSND: [num_blocks,block_size,1,D] / [..,Dv]
 *                  through block_table (a dense pool)
 *   dtype          LI_BF16 or LI_FP16 for query, key, value and out
 *   N1             query heads: 16, 32, 64 or 128
 *   D, Dv          128 and 128
 *   sparse_count   K, entries per index row, 1..65536
 *   softmax_scale  > 0 and finite (1/sqrt(D) is the usual choice)
 *   B, S1, S2, T1, T2, num_blocks, block_size, max_blocks_per_seq  as in li_params
 *   reserved       must be 0
 *
 *   sparse_indices int32 [rows, K] (the indexer's output layout): batch-local
 *                  key positions; -1 marks an empty slot.  An entry >= Sk_b or
 *                  below -1 is skipped and flagged with LI_DEV_BAD_INDEX.
 *   act_seq_q, act_seq_k, block_table   as for li_indexer
 *   out            [rows, N1, Dv] in dtype (device)
 *   lse            fp32 [rows, N1] (device) or NULL
 *   status         device int32 that receives LI_DEV_* bits by atomic OR, or
 *                  NULL; the caller clears it.  LI_DEV_BAD_INDEX: an entry
 *                  outside [-1, Sk_b) (skipped); LI_DEV_BAD_BLOCK: a
 *                  block_table entry outside [0, num_blocks) behind a valid
 *                  index (skipped); LI_DEV_TIMEOUT: a pipeline wait expired
 *                  (out and lse are then undefined; the kernel still ends)
 * Pointers: query, key, value and out 16-byte aligned; sparse_indices, lse and
 * status 4-byte aligned (else LI_ERR_SHAPE, nothing launched).
 * Accumulation is fp32 on the tensor cores; the softmax weights enter the P.V
 * product rounded to dtype.  Needs no workspace.  One launch (a thread-block
 * cluster per row when rows are few).
 */
#define LI_DEV_BAD_INDEX     0x20  /* sparse attention: an index outside [-1, Sk) (skipped) */
typedef struct {
    int32_t layout_q, layout_kv;
    int32_t dtype;
    int32_t B, S1, S2, T1, T2;
    int32_t N1, D, Dv;
    int32_t num_blocks, block_size, max_blocks_per_seq;
    int32_t sparse_count;
    float softmax_scale;
    int32_t reserved;
} li_sfa_params;

LI_API li_status li_sparse_attention(const li_sfa_params *p, const void *query, const void *key,
                                     const void *value, const int32_t *sparse_indices,
                                     const int32_t *act_seq_q, const int32_t *act_seq_k,
                                     const int32_t *block_table, void *out, float *lse,
                                     int32_t *status, void *stream);

/*
 * Rotary positions for the query and key heads that the indexer and the
 * attention read.  Pair p (0 <= p < rot_dim/2) of row r turns by the angle
 * a = positions[r] * inv_freq[p]:
 *
 *     y0 = mscale * (x0 cos a - x1 sin a)
 *     y1 = mscale * (x1 cos a + x0 sin a)          (inverse: sin a -> -sin a)
 *
 * with x0, x1 at columns rot_offset + p and rot_offset + p + rot_dim/2 of the
 * head (LI_ROPE_HALF) or rot_offset + 2p and rot_offset + 2p + 1
 * (LI_ROPE_INTERLEAVED).  The other columns are copied.  `inverse` is the
 * transposed turn: it undoes a call with the same mscale = 1, and for any
 * mscale it takes an output's gradient to the input's.
 *
 *   dtype         LI_BF16, LI_FP16 or LI_FP32: query, key and outputs
 *   rows          token rows (B*S1 or T1); 0 does nothing (the tensors' pointers
 *                 may then be NULL)
 *   N1, N2        query heads 1..1024; key heads 0..1024 (0: no key, key pointers NULL)
 *   D             head dim 2..1024
 *   rot_dim       even, 2..D; rot_offset >= 0; rot_offset + rot_dim <= D
 *   mscale        finite, > 0 (1 when positions are not scaled)
 *   *_stride      elements between consecutive rows / heads of query, key and
 *                 the outputs (0 = dense: N*D and D), so that heads may lie in
 *                 a wider projection; heads may not overlap (head stride >= D,
 *                 row stride >= (N-1)*head stride + D)
 *   reserved      must be 0
 *   positions     device int32 [rows], any value
 *   inv_freq      device fp64 [rot_dim/2], radians per position
 *                 (li_rope_frequencies); the angle is reduced in 64 bits, so a
 *                 far position costs no accuracy
 * An output may be its input (same strides); otherwise outputs overlap
 * nothing.  Pointers are aligned to their element; 16-byte alignment of
 * everything (pointers, strides, D, rot_offset, and rot_dim/2 for
 * LI_ROPE_HALF) is what the wide loads need.  One launch, no workspace.
 */
typedef enum { LI_ROPE_HALF = 0, LI_ROPE_INTERLEAVED = 1 } li_rope_pairing;
typedef struct {
    int32_t dtype;
    int32_t rows, N1, N2, D;
    int32_t rot_dim, rot_offset;
    int32_t pairing, inverse;
    float mscale;
    int64_t q_row_stride, q_head_stride, k_row_stride, k_head_stride;
    int64_t q_out_row_stride, q_out_head_stride, k_out_row_stride, k_out_head_stride;
    int32_t reserved;
} li_rope_params;

LI_API li_status li_rope(const li_rope_params *p, const int32_t *positions, const double *inv_freq,
                         const void *query, const void *key, void *query_out, void *key_out,
                         void *stream);

/*
 * Host only: the radians per position of each pair, into inv_freq[rot_dim/2]
 * (host memory), and the factor for li_rope_params.mscale.
 *   LI_ROPE_SCALE_NONE    base^(-2p/rot_dim)
 *   LI_ROPE_SCALE_LINEAR  the same / factor (positions interpolated)
 *   LI_ROPE_SCALE_NTK     base replaced by base * factor^(rot_dim/(rot_dim-2))
 *   LI_ROPE_SCALE_YARN    pairs that turn at least beta_fast times within
 *                         original_positions are kept, those that turn at most
 *                         beta_slow times are divided by factor, a linear ramp
 *                         over p lies between; mscale = 0.1 ln(factor) + 1
 * factor >= 1 (ignored by NONE); base > 1; rot_dim even, 2..1024 (NTK: >= 4);
 * YARN needs original_positions >= 1 and beta_fast > beta_slow > 0.
 */
typedef enum { LI_ROPE_SCALE_NONE = 0, LI_ROPE_SCALE_LINEAR = 1, LI_ROPE_SCALE_NTK = 2, LI_ROPE_SCALE_YARN = 3 } li_rope_scaling;
LI_API li_status li_rope_frequencies(int32_t scaling, int32_t rot_dim, double base, double factor,
                                     int32_t original_positions, double beta_fast, double beta_slow,
                                     double *inv_freq, float *mscale);

/*
 * The pages of a PA_BSND cache.  A cache is one or more pools (keys, values,
 * scales, of any number of layers) whose axis 0 is the page ("block" in the
 * calls that read them), a block_table [B, max_pages_per_seq], the lengths
 * act_seq_k [B] and a reference count per page [num_pages] (0 = free); row b
 * holds its pages in the first ceil(len_b / page_size) columns.  The calls
 * below take this state (table, lens, refs) and write the new one to table_out,
 * lens_out and refs_out, each of which is either its input (in place) or a
 * buffer that overlaps nothing.  All decisions are taken on the device, in an
 * order that does not depend on timing: free pages are handed out lowest page
 * first, rows and pairs are served in the order of the arguments.
 *
 *   li_pages_reserve  grows row b to new_lens[b] tokens (a length that is not
 *                     above the present one changes nothing)
 *   li_pages_fork     makes the empty row dst_rows[i] a child of src_rows[i]:
 *                     whole pages are shared (their count goes up), a partly
 *                     filled last page is copied into a fresh one, so a page
 *                     that is still written to has one owner
 *   li_pages_free     empties rows: each of their pages' counts goes down, the
 *                     row's columns become -1, its length 0
 *   li_pages_compact  moves live pages down so that the n live pages are the
 *                     pages 0 .. n-1: the i-th live page at or above n goes to
 *                     the i-th free page below n; columns behind a row's pages
 *                     become -1
 *   li_pages_copy     copies page src[i] to page dst[i] of every pool; the
 *                     destinations are distinct and no destination is a source
 *                     of another pair (else their contents are undefined)
 *
 * When the free pages run out, the rows (pairs) that need a fresh page are left
 * as they were from the first that no longer fits on, and LI_DEV_NO_PAGES is
 * flagged; those that need none (a row that grows inside its last page, a child
 * of whole pages) are served wherever they stand.  A row outside [0, B), a row
 * named twice (the first counts), a fork onto a row that is not empty: skipped,
 * LI_DEV_BAD_ROW.  A length outside [0, max_pages_per_seq *
 * page_size]: the present length is clamped, a new one skipped,
 * LI_DEV_BAD_KLEN.  A page number outside [0, num_pages), a page whose count
 * would fall below 0: skipped (-1 in a written row), LI_DEV_BAD_BLOCK.
 *
 *   num_pages 1..2^26; page_size, max_pages_per_seq, B >= 1; max_pages_per_seq *
 *   page_size and B * max_pages_per_seq <= 2^31-1
 *   pools      host array of n_pools (0..256) descriptors: base (device), bytes
 *              of one page, bytes between pages (>= page_bytes)
 *   status     device int32 that receives LI_DEV_* bits by atomic OR, or NULL
 *   workspace  device buffer of li_pages_workspace_size bytes, 256-byte
 *              aligned, not shared by calls that may run at the same time
 * Two launches (li_pages_copy: one; one more per 64 pools beyond the first 64).
 */
#define LI_DEV_NO_PAGES      0x40  /* pages: the free pages ran out (rows that need one left as they were) */
#define LI_DEV_BAD_ROW       0x80  /* pages: a row out of range, named twice, or not empty (skipped) */
typedef struct {
    int32_t num_pages, page_size, max_pages_per_seq, B;
    int32_t reserved;
} li_pages_params;
typedef struct {
    void *base;
    int64_t page_bytes, page_stride;
} li_page_pool;

LI_API li_status li_pages_workspace_size(const li_pages_params *p, size_t *bytes);
LI_API li_status li_pages_copy(const li_pages_params *p, const li_page_pool *pools, int32_t n_pools,
                               const int32_t *src_pages, const int32_t *dst_pages, int32_t n,
                               int32_t *status, void *stream);
LI_API li_status li_pages_reserve(const li_pages_params *p, const int32_t *table, const int32_t *lens,
                                  const int32_t *refs, const int32_t *new_lens, int32_t *table_out,
                                  int32_t *lens_out, int32_t *refs_out, int32_t *status,
                                  void *workspace, size_t workspace_bytes, void *stream);
LI_API li_status li_pages_fork(const li_pages_params *p, const li_page_pool *pools, int32_t n_pools,
                               const int32_t *table, const int32_t *lens, const int32_t *refs,
                               const int32_t *src_rows, const int32_t *dst_rows, int32_t n,
                               int32_t *table_out, int32_t *lens_out, int32_t *refs_out,
                               int32_t *status, void *workspace, size_t workspace_bytes, void *stream);
LI_API li_status li_pages_free(const li_pages_params *p, const int32_t *table, const int32_t *lens,
                               const int32_t *refs, const int32_t *rows, int32_t n, int32_t *table_out,
                               int32_t *lens_out, int32_t *refs_out, int32_t *status, void *workspace,
                               size_t workspace_bytes, void *stream);
LI_API li_status li_pages_compact(const li_pages_params *p, const li_page_pool *pools, int32_t n_pools,
                                  const int32_t *table, const int32_t *lens, const int32_t *refs,
                                  int32_t *table_out, int32_t *lens_out, int32_t *refs_out,
                                  int32_t *status, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Segment-sparse attention: attention over the segments of seg_size
 * consecutive keys that a cheap score selects for each query row and key head
 * (the coarse sibling of li_indexer + li_sparse_attention: one score per
 * segment instead of one per key, and any number of key heads).  With
 * vis(r) the keys that row r sees (sparse_mode 0: Sk; 3: right-down causal,
 * t <= i + Sk - Sq), ns(r) = ceil(vis(r) / seg_size) and n = the key head of
 * query head h (heads n*G .. n*G+G-1, G = N1/N2):
 *
 *   li_segment_pool       P[b,s,n] = mean of key[t,n] over the keys t of
 *                         segment s that lie below Sk
 *   li_segment_select     score(r,n,s) = (sum of q[r,h] over the heads of n) . P[b,s,n],
 *                         in 64 bits; the first init_segs and the last local_segs
 *                         of the ns(r) segments are always selected, the best
 *                         others fill the seg_count entries (ties: the lower
 *                         segment; NaN counts as -inf).  Selected segments are
 *                         written in ascending order, -1 behind them.
 *   li_segment_attention  J = keys t < vis(r) of the selected segments;
 *                         out_h = sum_J softmax(softmax_scale q_h . k_t) v_t,
 *                         lse_h = log sum_J exp(softmax_scale q_h . k_t);
 *                         0 and -inf when J is empty, for BSND padding rows and
 *                         for TND rows behind the last sequence (select: -1).
 *                         What a row does not select has no effect on it, not
 *                         even as a NaN or infinity.  (Time it does cost: results
 *                         that a value which is not finite reached, a row's own
 *                         or a neighbour's, are computed again key by key, about
 *                         0.36 us a key for each of a block's up to 128.)
 *
 *   layout_q, layout_kv   as li_sfa_params, with N2 key heads: key and value
 *                         [B,S2,N2,D], [T2,N2,D] or [num_blocks,block_size,N2,D]
 *   dtype                 LI_BF16 or LI_FP16: query, key, value, out
 *   N1, N2, D             N2 divides N1, G = N1/N2 <= 128, N1 <= 1024; D (also
 *                         the values' dim) 64 or 128
 *   block_size            pages: a multiple of 16
 *   kv_block_stride       elements between pages of the key pool and of the value
 *                         pool (0 = dense); a multiple of 8
 *   seg_size              a multiple of 16 in [16, 1024]
 *   seg_count             entries per (row, key head), 1..1024
 *   init_segs, local_segs >= 0, together <= seg_count; local_segs >= 1 with
 *                         sparse_mode 3 (a segment that a row sees in part is
 *                         then always selected and its mean, which looks ahead,
 *                         is never used)
 *   max_segs              segments per sequence of P: [B, max_segs, N2, D]
 *                         fp32; 1..16384.  Longer sequences are cut there and
 *                         flagged with LI_DEV_BAD_KLEN (pool and select only).
 *   softmax_scale         > 0 and finite
 *   reserved              must be 0
 *
 *   first      (pool) device int32 [B] or NULL: only the segments of tokens
 *              first[b] .. Sk-1 are written, as after appending tokens;
 *              segments before them and behind the last keep what they hold
 *   pooled     device fp32, 16-byte aligned
 *   seg_idx    int32 [rows, N2, seg_count]; attention takes ascending entries, -1
 *              anywhere is skipped; an entry that is below -1, not below
 *              ceil(Sk/seg_size), or not above the entries before it in its
 *              row is skipped and flagged with LI_DEV_BAD_INDEX
 *   out        [rows, N1, D] dtype; lse fp32 [rows, N1] or NULL
 *   status     as in li_sparse_attention
 * No query rows: select and attention do nothing.  No keys (S2 or T2 of 0):
 * pool does nothing, attention writes 0 and -inf.  Pointers of tensors without
 * elements may be NULL.
 * Pointers: query, key, value, out and pooled 16-byte aligned, the others
 * 4-byte.  Accumulation is fp32; the softmax weights enter the P.V product
 * rounded to dtype and out is divided by the sum of those (lse holds the sum of
 * the weights before rounding).  One launch each, no workspace.
 */
typedef struct {
    int32_t layout_q, layout_kv;
    int32_t dtype;
    int32_t B, S1, S2, T1, T2;
    int32_t N1, N2, D;
    int32_t num_blocks, block_size, max_blocks_per_seq;
    int64_t kv_block_stride;
    int32_t seg_size, seg_count, init_segs, local_segs, max_segs;
    int32_t sparse_mode;
    float softmax_scale;
    int32_t reserved;
} li_segment_params;

LI_API li_status li_segment_pool(const li_segment_params *p, const void *key, const int32_t *act_seq_k,
                                 const int32_t *block_table, const int32_t *first, float *pooled,
                                 int32_t *status, void *stream);
LI_API li_status li_segment_select(const li_segment_params *p, const void *query, const float *pooled,
                                   const int32_t *act_seq_q, const int32_t *act_seq_k, int32_t *seg_idx,
                                   int32_t *status, void *stream);
LI_API li_status li_segment_attention(const li_segment_params *p, const void *query, const void *key,
                                      const void *value, const int32_t *seg_idx,
                                      const int32_t *act_seq_q, const int32_t *act_seq_k,
                                      const int32_t *block_table, void *out, float *lse,
                                      int32_t *status, void *stream);

/* Thread-local message describing the last non-OK status. */
LI_API const char *li_last_error(void);

/*
 * SYNCHRONISING: copy the device status word of `workspace` to the host after
 * everything queued on `stream` has finished.  *flags receives the LI_DEV_*
 * bits of the last call that used this workspace.  Returns LI_ERR_DEVICE when
 * any bit is set, LI_OK otherwise.
 */
LI_API li_status li_read_device_status(const void *workspace, void *stream, int32_t *flags);

/*
 * Self-test of the bounded wait used by every pipeline barrier: one thread
 * waits on a shared-memory barrier that nothing will ever complete, gives up
 * after timeout_ns nanoseconds and ORs LI_DEV_TIMEOUT into *status_word (a
 * device int32).  Lets a test check that an expired wait reports an error and
 * leaves the context usable, without faulting or hanging the GPU.
 */
LI_API li_status li_selftest_bounded_wait(int32_t *status_word, int64_t timeout_ns, void *stream);

/*
 * Per-stage timing: when `events` holds n >= 4 cudaEvent_t handles (passed as
 * void*), every later li_indexer / li_quant_indexer call on this thread records
 * events[0] before the scheduler, events[1] after it, events[2] after the score
 * kernel and events[3] after the Top-k kernel, on the call's stream.  n = 0 or
 * events = NULL turns it off.  The handles are borrowed, not owned.
 */
LI_API void li_set_profile_events(void *const *events, int32_t n);

/* Number of kernels launched by the last successful call on this thread. */
LI_API int32_t li_last_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* LI_H */
