/*
 * fp8mla.h -- C ABI of libfp8mla.so: decode-phase attention over an FP8
 * (E4M3, OCP "fn" encoding) paged KV cache on sm_103a.
 *
 * Three variants of one operation, all "softmax(scale * q . k) @ v over the
 * keys of a paged cache", plus the bookkeeping around them:
 *
 *   fp8mla_get_metadata / fp8mla_decode  -- dense MLA decode: d = 576
 *       (512 latent + 64 RoPE), dv = 512 (V is the first 512 dims of the
 *       same cached row), one shared KV head, s_q = 1..2 query tokens with a
 *       bottom-right causal mask.  FlashMLA "update fp8 support":
 *       Improvements (FP8 Q and KV, Q.K over nine 64-wide K chunks with the
 *       RoPE chunk kept at 16 bit) and the H800 test shape (b, s_q, h_q,
 *       h_kv = 1, d = 576, dv = 512, causal).
 *   sparse_mla_decode -- top-k sparse MLA: each query token attends to the
 *       rows listed in its top-k index list of one flat cache (rope-free
 *       d = dv = 512).  aiter "Support fp8 KV caches and fp8 dots in
 *       sparse_mla_fwd on gfx942": Technical details (in-kernel Q
 *       quantisation, P quantised as p * 128 with the factor divided out in
 *       the epilogue) and Results (16 heads, top-k 2048).
 *   paged_gqa_decode -- grouped-query paged decode with separate K and V
 *       caches and split-KV flash-decoding.  InfiniCore "add FP8 blockwise
 *       dequantize/GEMM operators and FP8(E4M3) KV cache support in paged
 *       attention": Summary (FP8 decode kernel, split-kv with a combine
 *       kernel, the "auto" waves heuristic) and the split-kv commit
 *       (partial (max, sum_exp, weighted sum) triples, empty shards publish
 *       m = -inf, l = 0, acc = 0).
 *
 * and the step that fills the cache:
 *
 *   fp8_paged_cache_write -- quantise new bf16 K or V rows into an E4M3
 *       paged cache, with per-row scales amax / 448 or one given per-tensor
 *       scale.  InfiniCore page, Summary: the paged_caching write kernel.
 *
 * and what a decode step does around it, also over a cache held in 4 bits:
 *
 *   rotary_table / rotary_apply -- rotary positions of query and key heads.
 *   paged_kv_append -- a step's K and V into the cache, K rotated on the way.
 *   paged_cache_read -- cached rows back as bf16.
 *   paged_gqa_decode_fp4 -- grouped-query decode over the 4-bit cache.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every pointer argument that names a tensor is a DEVICE pointer unless
 *    stated otherwise; the caller owns all memory (inputs, outputs,
 *    workspace, metadata).  The library allocates nothing on these calls;
 *    it keeps only a small host-side cache of encoded TMA descriptors.
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *    default stream) and returns as soon as its kernels are enqueued.
 *  - Arguments are checked on the host before anything is launched; a bad
 *    argument returns a status and launches nothing.  Device-side problems
 *    (an index out of range, a bounded wait that ran out) never trap: the
 *    kernel records a bit in a device status word and skips the work;
 *    fp8mla_get_last_device_error() reads and clears it.
 *  - Values: the cache holds E4M3 bytes; true value = kv_scale * decode(byte)
 *    with one float32 per-tensor scale (amax / 448 on the InfiniCore page)
 *    passed as a DEVICE pointer to one float.  Q is bf16.  Outputs: bf16
 *    `out` and float32 `lse` = natural log of sum_j exp(scale * q . k_j).
 *  - A row that sees no key (empty cache, causal cut, all indices -1) gets
 *    out = 0 and lse = -inf (InfiniCore zero-length-row commit; FlashInfer
 *    "add xqa fp8 mha and fp8 kv cache", review of fully masked rows).
 *  - Cache bytes past a sequence's length and pages the block table does not
 *    reference are never read and may hold anything (NaN included).
 */
#ifndef FP8MLA_H
#define FP8MLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define FP8MLA_API __attribute__((visibility("default")))
#else
#define FP8MLA_API
#endif

typedef struct CUstream_st* fp8mla_stream_t; /* same type as cudaStream_t */

typedef enum {
  FP8MLA_OK = 0,
  FP8MLA_ERR_INVALID_ARG = 1,       /* null pointer, bad shape, missing kv scale, ... */
  FP8MLA_ERR_UNSUPPORTED_DTYPE = 2, /* cache encoding other than OCP E4M3 */
  FP8MLA_ERR_WORKSPACE_TOO_SMALL = 3,
  FP8MLA_ERR_CUDA = 4,              /* a CUDA runtime/driver call failed */
  FP8MLA_ERR_DEVICE = 5             /* not a launch failure: see fp8mla_get_last_device_error */
} fp8mla_status_t;

/* Precision of the two dot products (Q.K and P.V).
 *  FP8MLA_DOT_16BIT: "bf16 dots" on the aiter page: Q and P keep bf16's 8
 *    significant bits, K and V are the cache's exact E4M3 values.  Dense MLA
 *    computes them as two-term E4M3 dots: the latent part of Q (with a
 *    per-row power-of-two scale) and P (as 64 * p) each enter as hi + lo,
 *    hi = E4M3(x), lo = E4M3(x - hi); the RoPE part of Q.K is f16.
 *  FP8MLA_DOT_FP8:   the latent part of Q is quantised to E4M3 with a
 *    per-row power-of-two scale, the RoPE part of Q.K stays 16-bit (f16 in
 *    dense MLA; FlashMLA page, Improvements), and P is quantised as E4M3
 *    (64 * p in dense MLA, 128 * p in sparse MLA; aiter page, Technical
 *    details).
 *  The first-order effect of rounding Q on the LSE is corrected (dense MLA,
 *  both modes; sparse MLA). */
typedef enum { FP8MLA_DOT_16BIT = 0, FP8MLA_DOT_FP8 = 1 } fp8mla_dot_mode_t;

/* Encoding of the cache bytes.  Unless an entry point names the 4-bit cache
 * (FP8MLA_KV_E2M1) too, only FP8MLA_KV_E4M3 (OCP e4m3 "fn", or a
 * uint8 view of it) is accepted; the others are refused with
 * FP8MLA_ERR_UNSUPPORTED_DTYPE instead of being misread (aiter page,
 * Technical details: "a typed cache in the other arch's encoding is
 * refused"). */
typedef enum {
  FP8MLA_KV_E4M3 = 0,
  FP8MLA_KV_E4M3FNUZ = 1,
  FP8MLA_KV_E5M2 = 2,
  FP8MLA_KV_OTHER = 3,
  FP8MLA_KV_E2M1 = 4 /* the 4-bit cache: paged_kv_append, paged_cache_read and paged_gqa_decode_fp4 only */
} fp8mla_kv_dtype_t;

/* Type of the values rotary_apply turns. */
typedef enum { FP8MLA_BF16 = 0, FP8MLA_F16 = 1, FP8MLA_F32 = 2 } fp8mla_dtype_t;

/* Layout of a rotated part and what becomes of padding: rotary_apply, paged_kv_append. */
#define FP8MLA_ROTARY_INTERLEAVED 0x1 /* pairs (2i, 2i + 1), else (i, i + rot / 2) */
#define FP8MLA_ROTARY_ZERO_Q 0x2      /* q_out's rows of tokens without a position become zeros, else are left */
#define FP8MLA_ROTARY_ZERO_K 0x4      /* the same for k_out (rotary_apply only) */

/* Device status bits reported by fp8mla_get_last_device_error. */
#define FP8MLA_DEV_WAIT_TIMEOUT 0x1u   /* a bounded mbarrier wait ran out; the CTA stopped */
#define FP8MLA_DEV_BAD_PAGE 0x2u       /* block-table entry outside [0, num_pages) */
#define FP8MLA_DEV_BAD_SEQLEN 0x4u     /* seqlen < 0 or more pages than the block table row */
#define FP8MLA_DEV_BAD_INDEX 0x8u      /* top-k index outside [-1, num_tokens) */
#define FP8MLA_DEV_BAD_SLOT 0x10u      /* cache-write slot >= num_blocks * page_size */
#define FP8MLA_DEV_BAD_POSITION 0x20u  /* position >= the rows of the rotary table */

/* ------------------------------------------------------------------ MLA ---
 * Work units.  The dense MLA kernel runs one work unit per pair of SMs (the
 * two CTAs of a unit each own one half of dv).  fp8mla_metadata_units(n)
 * is the number of units for a GPU with n SMs: max(1, n / 2). */
FP8MLA_API int fp8mla_metadata_units(int num_sms);

/* fp8mla_get_metadata -- split the batch's (sequence, 64-token page) work
 * list into `num_units` contiguous page ranges of balanced cost (each page
 * costs 1, each (sequence, unit) segment a fixed 4 more).  Computed once per
 * decode step on the device, reused by every layer.
 *   cache_seqlens  int32 [b] (device)
 *   h_q, s_q       query heads and tokens (h_q * s_q <= 128)
 *   num_units      fp8mla_metadata_units(num_sms)
 *   force_splits   0 = balanced; k > 0 = cut every sequence into min(k,
 *                  pages) near-equal chunks, one unit each (needs
 *                  b * k <= num_units) -- for split-KV tests
 *   tile_sched     int32 [num_units][8] (device, written): {b_begin,
 *                  page_begin, b_end, page_end, split index of the first
 *                  segment, 0, 0, 0}; the range ends before (b_end, page_end)
 *   num_splits     int32 [b + 1] (device, written): prefix sum of the number
 *                  of units touching each sequence (0 for an empty one). */
FP8MLA_API fp8mla_status_t fp8mla_get_metadata(const int32_t* cache_seqlens, int b, int h_q, int s_q, int num_units,
                                    int force_splits, int32_t* tile_sched, int32_t* num_splits,
                                    fp8mla_stream_t stream);

/* Workspace of fp8mla_decode: (b + num_units) split-KV partial slots of
 * 128 x 512 bf16 accumulators plus 128 (m, l) pairs each, then per sequence
 * its quantised Q, the E4M3 hi term in both dot modes (88 064 bytes: the
 * decode kernel's Q slots), and 128 Q scales. */
FP8MLA_API size_t fp8mla_workspace_bytes(int b, int s_q, int h_q, int num_units);

/* fp8mla_decode -- dense MLA decode over the paged E4M3 cache.
 *   q              bf16 [b, s_q, h_q, 576]
 *   kv_cache       E4M3 bytes [num_pages, 64, 576]; row = 512 latent || 64 RoPE
 *   kv_dtype       must be FP8MLA_KV_E4M3
 *   block_table    int32 [b, max_pages]; logical page p of sequence i lives at
 *                  physical page block_table[i * max_pages + p]
 *   cache_seqlens  int32 [b]; keys per sequence (0 allowed)
 *   kv_scale       float32 [1] (device): per-tensor dequantisation scale; NULL
 *                  is refused (InfiniCore "F8 cache without scales fails
 *                  loudly (Bad Parameter)")
 *   softmax_scale  multiplier of q . k (e.g. 1/sqrt(576))
 *   causal         1: query token i of s_q sees keys j < s_k - s_q + i + 1
 *   tile_sched, num_splits, num_units -- from fp8mla_get_metadata on the same
 *                  cache_seqlens
 *   workspace      >= fp8mla_workspace_bytes(b, s_q, h_q, num_units) bytes,
 *                  256-byte aligned; contents need not be initialised
 *   out            bf16 [b, s_q, h_q, 512] (written)
 *   lse            float32 [b, s_q, h_q] (written)
 *   dot_mode       FP8MLA_DOT_FP8 or FP8MLA_DOT_16BIT
 * Requires h_q * s_q <= 128, kv_cache / q / out 16-byte aligned. */
FP8MLA_API fp8mla_status_t fp8mla_decode(const void* q, const void* kv_cache, fp8mla_kv_dtype_t kv_dtype, int num_pages,
                              const int32_t* block_table, int max_pages, const int32_t* cache_seqlens,
                              const float* kv_scale, float softmax_scale, int causal, const int32_t* tile_sched,
                              const int32_t* num_splits, int num_units, void* workspace, size_t workspace_bytes,
                              void* out, float* lse, fp8mla_dot_mode_t dot_mode, int b, int s_q, int h_q,
                              fp8mla_stream_t stream);

/* fp8mla_decode_ext -- fp8mla_decode with one dequantisation scale per cached
 * row (InfiniCore page, Summary: FP8 caches carry scales of shape
 * [num_blocks, num_kv_heads, block_size]; here one KV head, so [num_pages, 64]).
 *   kv_scale_rows  float32 [num_pages, 64] (device, 16-byte aligned) or NULL;
 *                  when set, row t of physical page p (its 512 latent and 64
 *                  RoPE values, K and V alike) is E4M3 code times
 *                  kv_scale_rows[p * 64 + t], every scale of a row a key uses
 *                  must be finite and not negative (below 2^-110 they count
 *                  as that for V, where a sequence's lie within a factor of
 *                  2^126), kv_scale is ignored (may be NULL), and only
 *                  FP8MLA_DOT_FP8 is accepted (FP8MLA_ERR_INVALID_ARG otherwise)
 *   kv_scale_rows NULL: exactly fp8mla_decode.
 * Other arguments, results and errors as fp8mla_decode. */
FP8MLA_API fp8mla_status_t fp8mla_decode_ext(const void* q, const void* kv_cache, fp8mla_kv_dtype_t kv_dtype,
                                             int num_pages, const int32_t* block_table, int max_pages,
                                             const int32_t* cache_seqlens, const float* kv_scale,
                                             const float* kv_scale_rows, float softmax_scale, int causal,
                                             const int32_t* tile_sched, const int32_t* num_splits, int num_units,
                                             void* workspace, size_t workspace_bytes, void* out, float* lse,
                                             fp8mla_dot_mode_t dot_mode, int b, int s_q, int h_q,
                                             fp8mla_stream_t stream);

/* ----------------------------------------------------------- sparse MLA ---
 * sparse_mla_decode -- query token t attends to the cache rows
 * topk_idx[t][0..topk) (an index of -1 is skipped), d = dv = 512 rope-free.
 *   q            bf16 [s_q, h_q, 512], 1 <= h_q <= 16 (the heads are the N
 *                dimension of one MMA tile); h_q > 16 -> FP8MLA_ERR_INVALID_ARG
 *   kv_cache     E4M3 bytes [num_tokens, 512], num_tokens < 2^31
 *   topk_idx     int32 [s_q, topk]; an index outside [-1, num_tokens) sets
 *                FP8MLA_DEV_BAD_INDEX and the key is skipped
 *   kv_scale     float32 [1] (device), NULL refused
 *   num_splits   0 = auto (about one CTA per SM over s_q tokens, at most one
 *                split per 128-key chunk), 1 = no split-K (one pass over all
 *                keys), k > 1 = keys cut into k contiguous shards merged by
 *                the combine step
 *   workspace    >= sparse_mla_workspace_bytes(s_q, h_q, topk, num_splits)
 *                bytes, 256-byte aligned; may be NULL when that is 0
 *   out          bf16 [s_q, h_q, 512]; lse float32 [s_q, h_q]
 *   dot_mode     must be FP8MLA_DOT_FP8 (Q quantised per row with a
 *                power-of-two scale, P as E4M3(128 p)); FP8MLA_DOT_16BIT is
 *                refused with FP8MLA_ERR_INVALID_ARG (this variant runs the
 *                aiter page's FP8-dot path only) */
FP8MLA_API fp8mla_status_t sparse_mla_decode(const void* q, const void* kv_cache, fp8mla_kv_dtype_t kv_dtype,
                                  int64_t num_tokens, const int32_t* topk_idx, int topk, const float* kv_scale,
                                  float softmax_scale, int num_splits, void* workspace, size_t workspace_bytes,
                                  void* out, float* lse, fp8mla_dot_mode_t dot_mode, int s_q, int h_q,
                                  fp8mla_stream_t stream);

/* Workspace bytes of sparse_mla_decode with these arguments: the split
 * partials of the split count the call will choose (auto uses the SM count
 * of the current device); 0 when that is a single split. */
FP8MLA_API size_t sparse_mla_workspace_bytes(int s_q, int h_q, int topk, int num_splits);

/* ------------------------------------------------------------------ GQA ---
 * paged_gqa_decode -- grouped-query decode; q head h reads KV head
 * h / (h_q / h_kv).
 *   q            bf16 [bs, h_q, head_dim]
 *   k_cache      E4M3 bytes [num_blocks, h_kv, page_size, head_dim]
 *   v_cache      E4M3 bytes [num_blocks, h_kv, page_size, head_dim]
 *   k_scale, v_scale  float32 [1] each (device), NULL refused
 *   block_table  int32 [bs, max_blocks]; seqlens int32 [bs]
 *   num_splits   0 = auto: when bs * h_kv CTAs already fill the GPU, every
 *                sequence is cut into a few key shards (about six CTAs per
 *                SM, at least 8 steps of 128 keys each, at most 16) so that
 *                unequal lengths balance; otherwise the fewest shards that
 *                fill the waves; k >= 1 forced
 *   workspace    >= paged_gqa_workspace_bytes(bs, h_q, head_dim, splits)
 *   out          bf16 [bs, h_q, head_dim]; lse float32 [bs, h_q]
 * Requires head_dim == 128, page_size == 16, h_q % h_kv == 0, h_q / h_kv <= 16. */
FP8MLA_API fp8mla_status_t paged_gqa_decode(const void* q, const void* k_cache, const void* v_cache,
                                 fp8mla_kv_dtype_t kv_dtype, int num_blocks, const float* k_scale,
                                 const float* v_scale, const int32_t* block_table, int max_blocks,
                                 const int32_t* seqlens, float softmax_scale, int num_splits, void* workspace,
                                 size_t workspace_bytes, void* out, float* lse, int bs, int h_q, int h_kv,
                                 int head_dim, int page_size, fp8mla_stream_t stream);

/* paged_gqa_decode_ext -- paged_gqa_decode with per-row KV scales and the XQA
 * options (FlashInfer "add xqa fp8 mha and fp8 kv cache": launcher arguments
 * for speculative decoding, sliding window and attention sinks; InfiniCore
 * page, Summary: scales of shape [num_blocks, num_kv_heads, block_size]).
 *   q            bf16 [bs, q_len, h_q, head_dim]: q_len query tokens per
 *                sequence, taken to be its last q_len cache positions (token i
 *                at position s_k - q_len + i)
 *   k_scale, v_scale  float32 [1] each, or with scale_per_row != 0 one float
 *                per cached row, [num_blocks, h_kv, page_size], 16-byte aligned,
 *                finite, not negative; V's below 2^-110 count as 2^-110, and
 *                a sequence's lie within a factor of 2^126
 *   spec_mask    uint8 [bs, q_len, q_len] (device) or NULL: token i sees key
 *                s_k - q_len + c of its own block iff spec_mask[b][i][c] != 0;
 *                NULL = causal inside the block (c <= i).  Keys before the
 *                block are always visible.
 *   window       0 = off; W > 0 keeps only keys j with (s_k - q_len + i) - j < W
 *   sinks        float32 [h_q] (device) or NULL: head h's softmax denominator
 *                gains e^{sinks[h]} (a key without value; -inf = no sink)
 *   out          bf16 [bs, q_len, h_q, head_dim]; lse float32 [bs, q_len, h_q]
 * A row that sees no key gets out = 0 and lse = its sink (-inf without one).
 * Requires q_len >= 1 and q_len * (h_q / h_kv) <= 16, window >= 0, and the
 * other requirements of paged_gqa_decode; workspace as paged_gqa_decode's.
 * Auto splits: paged_gqa_ext_num_splits (with a window, a grid that fills the
 * GPU is not split; never more shards than paged_gqa_num_splits gives, so its
 * workspace size suffices). */
FP8MLA_API fp8mla_status_t paged_gqa_decode_ext(const void* q, const void* k_cache, const void* v_cache,
                                                fp8mla_kv_dtype_t kv_dtype, int num_blocks, const float* k_scale,
                                                const float* v_scale, int scale_per_row, const int32_t* block_table,
                                                int max_blocks, const int32_t* seqlens, float softmax_scale, int q_len,
                                                const uint8_t* spec_mask, int window, const float* sinks,
                                                int num_splits, void* workspace, size_t workspace_bytes, void* out,
                                                float* lse, int bs, int h_q, int h_kv, int head_dim, int page_size,
                                                fp8mla_stream_t stream);

FP8MLA_API size_t paged_gqa_workspace_bytes(int bs, int h_q, int head_dim, int max_splits);

/* Number of key shards paged_gqa_decode will use for these arguments
 * (num_splits as passed: 0 = auto).  Host-only, no device access. */
FP8MLA_API int paged_gqa_num_splits(int bs, int h_kv, int max_seqlen, int num_sms, int num_splits);

/* Number of key shards paged_gqa_decode_ext will use: paged_gqa_num_splits's
 * rule, except that with a window (window > 0) max_seqlen is taken as the
 * keys the window spans (window + q_len - 1 + 128 at most) and a grid of
 * bs * h_kv CTAs that already fills the GPU is not split (the window makes
 * the sequences' work nearly equal); never more than paged_gqa_num_splits
 * gives for the same arguments.  Host-only. */
FP8MLA_API int paged_gqa_ext_num_splits(int bs, int h_kv, int max_seqlen, int q_len, int window, int num_sms,
                                        int num_splits);

/* ---------------------------------------------------------- cache write ---
 * fp8_paged_cache_write -- quantise-on-write of new K or V rows into an E4M3
 * paged cache (InfiniCore "add FP8 blockwise dequantize/GEMM operators and
 * FP8(E4M3) KV cache support in paged attention", Summary, paged_caching: a
 * write kernel over (token, kv_head) rows; per-row scale amax / 448, 1 when
 * amax is 0, kept in a float32 [num_blocks, h_kv, page] array).
 *   x             bf16 (device): the row of token t, head h starts at element
 *                 t * x_token_stride + h * head_dim and holds head_dim values;
 *                 x 16-byte aligned, x_token_stride a multiple of 8 and
 *                 >= h_kv * head_dim
 *   slot_mapping  int32 [n_tokens] (device): token t goes to block
 *                 slot / page_size, offset slot % page_size.  A negative slot
 *                 skips the token; a slot >= num_blocks * page_size sets
 *                 FP8MLA_DEV_BAD_SLOT and skips it.  Two tokens with the same
 *                 slot race: which one lands is undefined.
 *   cache         E4M3 bytes [num_blocks, h_kv, page_size, head_dim] (device,
 *                 16-byte aligned).  The dense MLA cache [num_pages, 64, 576]
 *                 is h_kv = 1, page_size = 64, head_dim = 576.
 *   exactly one of
 *     tensor_scale  float32 [1] (device): code = E4M3(fp32(x * inv)) with
 *                   inv = fp32(1 / tensor_scale); the value must be a normal
 *                   float > 0 (it is not read on the host)
 *     token_scales  float32 [num_blocks, h_kv, page_size] (device): each
 *                   written row gets scale = fp32(max|x| / 448) (1.0 when the
 *                   row is all zeros), stored at its slot, and
 *                   code = E4M3(fp32(x * inv)) with inv = fp32(448 / max|x|)
 *                   (1.0 for a zero row); a row with max|x| < 2^-64 is first
 *                   multiplied by 2^64 (exact), so inv stays finite
 * Every float operation rounds to nearest even; E4M3 rounding is to nearest
 * even with saturation to +-448.  x must be finite.  head_dim is a multiple
 * of 8 in [8, 1024]; kv_dtype must be FP8MLA_KV_E4M3.  n_tokens = 0 is a
 * no-op.  Bytes and scales of slots no token maps to are not touched.
 * Asynchronous on `stream`; the caller owns every buffer. */
FP8MLA_API fp8mla_status_t fp8_paged_cache_write(const void* x, int64_t x_token_stride, const int32_t* slot_mapping,
                                                 int n_tokens, int h_kv, int head_dim, int page_size,
                                                 int num_blocks, fp8mla_kv_dtype_t kv_dtype, void* cache,
                                                 const float* tensor_scale, float* token_scales,
                                                 fp8mla_stream_t stream);

/* --------------------------------------------------------------- rotary ---
 * A pair (a, b) of a head at position p turns by the angle p * inv_freq[i]:
 *   (a c - b s, b c + a s),  c = factor cos(angle), s = factor sin(angle).
 * Pair i of the rotated part (rot dims from rot_offset) is its dims
 * (i, i + rot / 2), or (2i, 2i + 1) when interleaved.  Scaling for long
 * contexts is a matter of inv_freq and factor.
 *
 * rotary_table -- table[p][i] = (cos, sin) of p * inv_freq[i], times factor.
 *   inv_freq  float64 [half] (device)
 *   table     float32 [n_positions, half, 2] (device, written); angles, cosines
 *             and sines are computed in 64 bits and rounded once
 * Requires 1 <= half <= 4096, factor > 0.  n_positions = 0 is a no-op. */
FP8MLA_API fp8mla_status_t rotary_table(const double* inv_freq, int half, int64_t n_positions, double factor,
                                        float* table, fp8mla_stream_t stream);

/* rotary_apply -- rotate the heads of q and (h_k > 0) of k.
 *   q, k          dtype [n_tokens, heads, head_dim], token and head strides in
 *                 elements, the dims of a head contiguous
 *   q_out, k_out  the same shapes with strides of their own; may be q and k
 *                 (in place).  Else no row of an output may overlap another
 *                 row or an input (refused; so are tensors of different
 *                 strides whose extents meet)
 *   positions     int32 or (positions_64 != 0) int64 [n_tokens] (device)
 *   table         float32 [n_positions, rot / 2, 2], 8-byte aligned
 *   layout        FP8MLA_ROTARY_* bits
 *   inverse       1: turn by the negative angle (the transpose: the gradient of
 *                 the rotation, and its inverse where factor is 1)
 * Every value is computed in float32 (products and sum each rounded) and
 * rounded once; dims outside the rotated part are copied.  A token with a
 * negative position is padding: its heads are not written.  A position >=
 * n_positions sets FP8MLA_DEV_BAD_POSITION and its heads are not written.  (Or
 * both become zeros: see layout.)
 * Requires 2 <= head_dim <= 8192, rot even, rot_offset + rot <= head_dim.  Any
 * stride and alignment of the type works; 16-byte aligned tensors whose
 * strides and rot_offset are multiples of 8 and rot of 16 go 8 pairs at a time. */
FP8MLA_API fp8mla_status_t rotary_apply(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                                        int64_t q_out_token_stride, int64_t q_out_head_stride, int h_q, const void* k,
                                        int64_t k_token_stride, int64_t k_head_stride, void* k_out,
                                        int64_t k_out_token_stride, int64_t k_out_head_stride, int h_k,
                                        fp8mla_dtype_t dtype, const void* positions, int positions_64,
                                        const float* table, int64_t n_positions, int n_tokens, int head_dim, int rot,
                                        int rot_offset, int layout, int inverse, fp8mla_stream_t stream);

/* ---------------------------------------------------------- 4-bit cache ---
 * A cached row of head_dim values is head_dim / 2 bytes of E2M1 codes (sign,
 * 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6; the even
 * dimension in the low nibble) and head_dim / 16 E4M3 block scales, with one
 * float32 scale for the whole cache:
 *   value = scale * s8[d / 16] * E2M1(code[d]).
 * codes [num_blocks, h_kv, page_size, head_dim / 2], block scales
 * [num_blocks, h_kv, page_size, head_dim / 16], both 16-byte aligned.  A
 * calibrated scale is amax / (448 * 6).
 *
 * paged_kv_append -- a step's new K and V rows into their slots, K rotated on
 * the way; optionally the step's queries rotated along.
 *   k, v          bf16 [n_tokens, h_kv, head_dim] (strides in elements,
 *                 multiples of 8; 16-byte aligned).  v and v_cache NULL: one
 *                 cache only (the dense MLA cache is h_kv = 1, page 64, 576)
 *   slot_mapping  int32 [n_tokens]: as fp8_paged_cache_write (a negative slot
 *                 skips the token's K and V)
 *   positions     int32 or int64 [n_tokens], with table.  A negative position
 *                 is padding: nothing of the token is written; one >=
 *                 n_positions sets FP8MLA_DEV_BAD_POSITION, likewise
 *   table         as rotary_apply's, 16-byte aligned; NULL: no rotation (then
 *                 q is NULL and positions are not read)
 *   kv_dtype      FP8MLA_KV_E4M3: k_scale (one float32, written codes are
 *                 E4M3(x fp32(1 / scale))) or k_row_scales (float32
 *                 [num_blocks, h_kv, page_size], written: amax / 448), exactly
 *                 one of them; FP8MLA_KV_E2M1: k_scale and k_block_scales
 *                 (written).  The same for v
 *   q, q_out      bf16 [n_tokens, h_q, head_dim] or NULL; q_out contiguous,
 *                 rotated like K; may be q.  A token without a position
 *                 leaves its rows, or zeros them (layout)
 * What is written (caches, scales, q_out) overlaps nothing else (refused).
 * The rotated row is quantised from float32.  E4M3 rows follow
 * fp8_paged_cache_write's arithmetic; an E2M1 block stores
 * s8 = E4M3(amax * fp32(1 / fp32(6 scale))) and codes
 * E2M1(x * fp32(1 / fp32(s8 scale))), 0 where s8 is 0.  Rounding is to nearest
 * even with saturation.  Rows must be finite, with two exceptions: an infinity
 * saturates (not with row scales), and a NaN is stored as NaN, in E2M1 in its
 * block's scale.  Scales are normal floats > 0 for which 6 * 448 * scale and
 * scale / 512 are normal too.  Two tokens with one
 * slot race.  Requires num_blocks * page_size < 2^31 (slots), n_tokens * heads
 * < 2^31 and head_dim a multiple of 16 in [16, 1024]; with a table
 * rot a multiple of 16 and rot_offset of 8 (of 16 when interleaved); in E2M1
 * with the half layout rot a multiple of 32 and rot_offset of 16. */
FP8MLA_API fp8mla_status_t paged_kv_append(
    const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
    int64_t v_head_stride, const int32_t* slot_mapping, int n_tokens, int h_kv, int head_dim, int page_size,
    int num_blocks, fp8mla_kv_dtype_t kv_dtype, void* k_cache, void* v_cache, const float* k_scale,
    const float* v_scale, float* k_row_scales, float* v_row_scales, void* k_block_scales, void* v_block_scales,
    const void* positions, int positions_64, const float* table, int64_t n_positions, int rot, int rot_offset,
    int layout, const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out, int h_q,
    fp8mla_stream_t stream);

/* paged_cache_read -- rows of a paged cache as bf16: out[i][h] is the row of
 * slot slots[i], KV head h, dequantised in float32 and rounded once.
 *   scales        as paged_kv_append: scale, row_scales, or scale and
 *                 block_scales (E2M1)
 *   out           bf16 [n, h_kv, head_dim], 16-byte aligned.  A negative slot
 *                 gives zeros; one past the cache too, with FP8MLA_DEV_BAD_SLOT.
 *                 Overlaps neither the cache nor its scales (refused)
 * head_dim a multiple of 8 (16 for E2M1) up to 1024, num_blocks * page_size and
 * n * h_kv < 2^31. */
FP8MLA_API fp8mla_status_t paged_cache_read(const void* cache, fp8mla_kv_dtype_t kv_dtype, const float* scale,
                                            const float* row_scales, const void* block_scales, const int32_t* slots,
                                            int n, int h_kv, int head_dim, int page_size, int num_blocks, void* out,
                                            fp8mla_stream_t stream);

/* paged_gqa_decode_fp4 -- paged_gqa_decode_ext over 4-bit caches.
 *   q            bf16 [bs, q_len, h_q, head_dim], 16-byte aligned
 *   k_cache, v_cache, k_block_scales, v_block_scales  as above
 *   k_scale, v_scale  float32 [1] each (device)
 *   block_table, seqlens, spec_mask, window, sinks, out, lse  as
 *                paged_gqa_decode_ext
 *   num_splits   0 = auto: one CTA, or a cluster of two, four or eight, per
 *                (sequence, KV head) where the block table holds few keys (from
 *                about 1000 up with few sequences, more as they come to fill the
 *                GPU), one CTA where the sequences fill it many times
 *                over, else the keys of all sequences cut into equal pieces,
 *                one per CTA that fits on the GPU; 1 = one CTA each; k > 1 =
 *                every sequence in k shards, at most one per 128 keys of the
 *                block table (the way to cut one long context among very many
 *                short ones, which auto leaves whole)
 *   workspace    >= paged_gqa_fp4_workspace_bytes with max_seqlen the block
 *                table's max_blocks * page_size, 256-byte aligned; may be
 *                NULL when that is 0
 *   out may be q; out, lse, workspace and q do not overlap otherwise (refused)
 * Products take K and V exactly, Q's values from 2^-31 of a head's largest on
 * exactly (others to 2^-39 of it); P is rounded to f16.  A NaN
 * reaches the rows that see its key, and those alone.  Scores and sinks may be
 * of any size that float32 holds in units of log2.
 * Scales are normal floats > 0.  Requires head_dim 64, 128 or 256, page_size
 * 16, 32, 64, 128 or 256, q_len <= 16, h_q % h_kv == 0, q_len * (h_q / h_kv)
 * <= 128 and fewer than 2^32 rows (num_blocks * h_kv * page_size) a cache. */
FP8MLA_API fp8mla_status_t paged_gqa_decode_fp4(const void* q, const void* k_cache, const void* v_cache,
                                                const void* k_block_scales, const void* v_block_scales, int num_blocks,
                                                const float* k_scale, const float* v_scale,
                                                const int32_t* block_table, int max_blocks, const int32_t* seqlens,
                                                float softmax_scale, int q_len, const uint8_t* spec_mask, int window,
                                                const float* sinks, int num_splits, void* workspace,
                                                size_t workspace_bytes, void* out, float* lse, int bs, int h_q,
                                                int h_kv, int head_dim, int page_size, fp8mla_stream_t stream);

/* Workspace bytes of paged_gqa_decode_fp4 with these arguments (auto uses the
 * SM count of the current device); 0 where nothing has to be merged. */
FP8MLA_API size_t paged_gqa_fp4_workspace_bytes(int bs, int h_q, int h_kv, int head_dim, int q_len,
                                                int64_t max_seqlen, int window, int num_splits);

/* ------------------------------------- many rows to paged E4M3 keys ---
 * paged_cross_attention -- attention of each sequence's query tokens to all
 * keys of that sequence's pages, whose number is independent of the tokens'
 * (an encoder's states, a document, a shared prefix):
 *   out[i, h] = softmax_j(softmax_scale q[i, h] . k_j) v_j over the kv_lens[b]
 *   keys of token i's sequence b, KV head h / (h_q / h_kv).
 *   q            bf16 [n_tokens, h_q, head_dim], strided along tokens and heads
 *                (elements, multiples of 8), 16-byte aligned; so is out
 *   k_cache, v_cache  E4M3 [num_blocks, h_kv, page_size, head_dim], 16-byte
 *                aligned; k_scale, v_scale float32 [1] (2^-80 to 2^80), or
 *                [num_blocks, h_kv, page_size] (16-byte aligned; 0 to 2^80)
 *                with scale_rows
 *   q_starts     int32 [bs + 1], not falling: sequence b has the tokens
 *                [q_starts[b], q_starts[b + 1]); NULL: token b (n_tokens >= bs)
 *   block_table  int32 [bs, max_blocks] (NULL where max_blocks is 0: no keys);
 *                kv_lens int32 [bs], 0 allowed
 *   out, lse     bf16, float32 [n_tokens, h_q] contiguous (natural log).  A
 *                sequence without keys gives zeros and -inf.  Rows of tokens of
 *                no sequence are left as they are, or get zeros (fill_out) and
 *                -inf (fill_lse)
 *   workspace    >= paged_cross_workspace_bytes, 256-byte aligned
 * out may be q (strided alike); out, lse and workspace overlap nothing else
 * (refused).  A length or token range that does not fit sets
 * FP8MLA_DEV_BAD_SEQLEN and counts as empty, a page outside the cache
 * FP8MLA_DEV_BAD_PAGE.  Products take K and V exactly, Q's values from 2^-9.8 of
 * a row's largest on exactly (others to 2^-17.8 of it); P is rounded to f16, sums
 * are float32.  A NaN reaches the rows of its sequence, and those alone.
 * Requires head_dim 64 or 128, page_size 16, 32, 64, 128 or 256, h_q % h_kv == 0,
 * h_q <= 65536, n_tokens * h_q <= 2^30, max_blocks * page_size <= 2^30,
 * bs <= 2^26 (with n_prefixes, below), fewer than 2^31 rows (num_blocks * h_kv *
 * page_size) a cache. */
FP8MLA_API fp8mla_status_t paged_cross_attention(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_cache, const void* v_cache,
    fp8mla_kv_dtype_t kv_dtype, int num_blocks, const float* k_scale, const float* v_scale, int scale_rows,
    const int32_t* q_starts, const int32_t* block_table, int max_blocks, const int32_t* kv_lens, float softmax_scale,
    void* workspace, size_t workspace_bytes, void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
    int fill_out, int fill_lse, int n_tokens, int bs, int h_q, int h_kv, int head_dim, int page_size,
    fp8mla_stream_t stream);

/* Workspace bytes of paged_cross_attention on the current device; max_keys =
 * max_blocks * page_size.  0 for sizes it refuses. */
FP8MLA_API size_t paged_cross_workspace_bytes(int n_tokens, int bs, int h_q, int h_kv, int head_dim, int64_t max_keys);

/* paged_gqa_decode_shared -- a decode step of sequences that share prefixes:
 * each of the n_prefixes prefixes is cached once, and its keys are read once
 * for all its sequences.  A row sees its prefix's keys, then its sequence's
 * own ones; positions are the caller's business (rotated when appended).
 *   q            bf16 [bs, q_len, h_q, head_dim], the last q_len own positions
 *   prefix_table int32 [n_prefixes, prefix_blocks], prefix_lens int32
 *                [n_prefixes] (0 allowed), prefix_starts int32 [n_prefixes + 1],
 *                not falling: prefix g belongs to the sequences
 *                [prefix_starts[g], prefix_starts[g + 1]); others have none
 *   block_table  int32 [bs, max_blocks], seqlens int32 [bs]: own keys, the
 *                step's q_len ones included; 0 allowed.  A table without columns
 *                is NULL here too
 *   spec_mask, sinks, out, lse  as paged_gqa_decode_ext (block key x of a
 *                sequence is its own key seqlens - q_len + x; one that would
 *                lie before key 0 does not exist)
 *   workspace    >= paged_gqa_shared_workspace_bytes, 256-byte aligned
 * The rest as paged_cross_attention; a NaN in the block's keys reaches only the
 * rows that see it.  q_len <= 32. */
FP8MLA_API fp8mla_status_t paged_gqa_decode_shared(
    const void* q, const void* k_cache, const void* v_cache, fp8mla_kv_dtype_t kv_dtype, int num_blocks,
    const float* k_scale, const float* v_scale, int scale_rows, const int32_t* prefix_table, int prefix_blocks,
    const int32_t* prefix_lens, const int32_t* prefix_starts, int n_prefixes, const int32_t* block_table, int max_blocks,
    const int32_t* seqlens, float softmax_scale, int q_len, const uint8_t* spec_mask, const float* sinks,
    void* workspace, size_t workspace_bytes, void* out, float* lse, int bs, int h_q, int h_kv, int head_dim,
    int page_size, fp8mla_stream_t stream);

/* Workspace bytes of paged_gqa_decode_shared on the current device, with the
 * tables' keys (blocks * page_size).  0 for sizes it refuses. */
FP8MLA_API size_t paged_gqa_shared_workspace_bytes(int bs, int q_len, int h_q, int h_kv, int head_dim, int n_prefixes,
                                                   int64_t max_prefix_keys, int64_t max_keys);

/* attention_merge -- joins attention results over disjoint keys, as the calls
 * of this header return them:
 *   lse = log sum_p exp(lses[p]), out = sum_p exp(lses[p] - lse) outs[p].
 *   outs         host array of `parts` device pointers, bf16 [n_tokens, heads,
 *                dim] strided along tokens and heads (host arrays of strides in
 *                elements, multiples of 8), 16-byte aligned; so is out
 *   lses         host array of device pointers, float32 [n_tokens, heads]
 * A part whose lse is -inf does not count, whatever its row holds; no part:
 * zeros and -inf.  An lse of NaN or +inf gives NaN in both.  Sums in float32,
 * rounded once.  out may be one of outs (strided alike); out and lse overlap
 * nothing else (refused).
 * 1 <= parts <= FP8MLA_MERGE_MAX_PARTS, dim a multiple of 8 up to 1024,
 * n_tokens * heads * dim <= 2^33. */
#define FP8MLA_MERGE_MAX_PARTS 8
FP8MLA_API fp8mla_status_t attention_merge(const void* const* outs, const int64_t* out_token_strides,
                                           const int64_t* out_head_strides, const float* const* lses, int parts,
                                           void* out, int64_t token_stride, int64_t head_stride, float* lse,
                                           int n_tokens, int heads, int dim, fp8mla_stream_t stream);

/* ------------------------------------------------------ no allocation ---
 * fp8mla_decode_no_alloc -- the dense MLA decode for callers that cannot
 * allocate device memory: code running where cudaMalloc is not allowed or
 * not available (inside a host runtime that only hands out fixed input and
 * output buffers, a plugin without access to an allocator, a process with
 * a hard memory budget fixed at start-up).  The pages have no counterpart:
 * this is a deployment convenience of this library.
 *
 * Same arguments and results as fp8mla_decode without the schedule and the
 * workspace: the call schedules one work unit per sequence (no split-KV) and
 * keeps its schedule, split counts and quantised Q in a fixed
 * device array compiled into this library (5.7 MB, held by every GPU that
 * loads the library until the process exits).  It calls no allocator.
 *   b <= FP8MLA_NO_ALLOC_MAX_BATCH; a larger batch returns
 *   FP8MLA_ERR_WORKSPACE_TOO_SMALL and launches nothing.
 *   All calls on a device share the array and it keeps the last call's
 *   contents (every call rewrites what it reads, so nothing needs clearing);
 *   calls that overlap on the GPU (other streams, other host threads) race on
 *   it, so the caller must serialise them.
 *   The first call on each device looks up the array's device address with
 *   that device current (cudaGetSymbolAddress); make that first call before
 *   capturing a stream into a graph. */
#define FP8MLA_NO_ALLOC_MAX_BATCH 64
FP8MLA_API fp8mla_status_t fp8mla_decode_no_alloc(const void* q, const void* kv_cache, fp8mla_kv_dtype_t kv_dtype,
                                                  int num_pages, const int32_t* block_table, int max_pages,
                                                  const int32_t* cache_seqlens, const float* kv_scale,
                                                  float softmax_scale, int causal, void* out, float* lse,
                                                  fp8mla_dot_mode_t dot_mode, int b, int s_q, int h_q,
                                                  fp8mla_stream_t stream);

/* ------------------------------------------------------- measurement ---- */

/* Stage timing of fp8mla_decode, a measurement aid (off by default).  While
 * enabled, fp8mla_decode records CUDA events before and after each of its
 * kernels (Q quantisation, the decode kernel, the combine);
 * those events keep the kernels from overlapping one another, so time the
 * call itself with timing off.  One timer per process, used by one thread at
 * a time: a decode call that times holds it for the call.  Enabling or
 * disabling discards the last record.  Returns FP8MLA_OK. */
FP8MLA_API fp8mla_status_t fp8mla_set_stage_timing(int enable);

/* Synchronises `stream` and writes ms[0..2] = milliseconds of the last timed
 * fp8mla_decode call's Q quantisation, decode kernel and
 * combine.  ms: host pointer to 3 floats.  FP8MLA_ERR_INVALID_ARG if no call
 * was timed since timing was enabled; FP8MLA_ERR_CUDA if the events cannot be
 * read (for instance when the last timed call ran on another device). */
FP8MLA_API fp8mla_status_t fp8mla_get_stage_times(fp8mla_stream_t stream, float* ms);

/* ------------------------------------------------------------- status ---- */

/* Synchronises `stream`, returns in *code_out the OR of the FP8MLA_DEV_* bits
 * recorded since the last call on the current device, and clears them. */
FP8MLA_API fp8mla_status_t fp8mla_get_last_device_error(fp8mla_stream_t stream, uint32_t* code_out);

/* Diagnostics of FP8MLA_DEV_WAIT_TIMEOUT in the dense MLA decode: synchronises
 * `stream` and writes where[0..2] = {source line of the wait, block index,
 * thread index} of the first bounded wait that ran out since the last call
 * on the current device (all 0 if none ran out), then clears the record.
 * where: host pointer to 3 uint32_t. */
FP8MLA_API fp8mla_status_t fp8mla_get_wait_timeout_site(fp8mla_stream_t stream, uint32_t* where);

/* Test hook of the bounded waits (FP8 dot mode of fp8mla_decode and
 * fp8mla_decode_no_alloc; paged_cross_attention and paged_gqa_decode_shared),
 * for the current device.  fault_page = p + 1 makes CTA 0 of work unit 0 of
 * every later FP8-dots decode skip the loads of the p-th page of its unit, so
 * the waits on that page run out: the decode then finishes with
 * FP8MLA_DEV_WAIT_TIMEOUT recorded (fp8mla_get_last_device_error) and wrong
 * values in that unit's outputs, and the CUDA context stays usable.  Cross
 * attention and shared prefixes: CTA 0 skips the p-th tile of 128 keys of K
 * that it meets, and the rows of its items from there on are wrong.
 * fault_page = 0 turns the hook off.  wait_limit_ns sets how long a bounded
 * wait may see no progress before it gives up (0 = the default: 4 s, there 3.5).
 * Not for production use; returns FP8MLA_ERR_CUDA if the symbols cannot be
 * written, FP8MLA_ERR_INVALID_ARG if fault_page < 0. */
FP8MLA_API fp8mla_status_t fp8mla_set_wait_test(int32_t fault_page, uint64_t wait_limit_ns);

/* Static string naming a status code. */
FP8MLA_API const char* fp8mla_status_string(fp8mla_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* FP8MLA_H */
