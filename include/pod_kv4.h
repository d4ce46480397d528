/*
 * pod_kv4.h -- C ABI of the 4-bit KV cache in libpod_attn.so: the steps around
 * the attention of pod_attn.h for a cache that holds K and V in 4 bits.
 *
 *   pod_qk_norm_rope  per-head RMS norm of q and k and the position rotation
 *   pod_kv4_write     quantises rows of K and V into the cache
 *   pod_kv4_read      reads rows back (what pod_attn_prefill_only then takes)
 *   pod_kv4_decode    single-token GQA attention over the cache (the 4-bit
 *                     counterpart of pod_attn_decode_only)
 *
 * The cache. Pages of 16 tokens; the pool is [pool_blocks, Hk, record] bytes,
 * one record for each (page, KV head), found through an int32 block table as
 * in pod_attn.h. Each channel group (32, 64 or 128 channels of one token of
 * one head, of K or of V) is held as 4-bit codes n with a pair (s, m) in fp16
 * and stands for n * s + m:
 *
 *     s = fp16((hi - lo) / 15), m = fp16(lo),
 *     n = min(max(rint((x - m) / s), 0), 15)     (n = 0 where s = 0)
 *
 * with lo, hi the group's least and largest value, the difference, its
 * fifteenth and the quotient rounded to fp32. (In fp16 rows s is one fp16 step
 * lower where m + 15 s would round to infinity, at 65520 and above.) Values beyond +-65504 are
 * cut to it. A group that holds an infinity or a NaN gets s = m = NaN: it
 * reads back as NaN throughout, and attention over it gives NaN. Where hi - lo
 * is below about 1e-3 the spacing of small fp16 numbers (2^-24) adds up to
 * 15 * 2^-25 to the error of half a step.
 *
 * A record holds, one after the other, d = head_dim, c = channel / 32,
 * the low four bits of a byte first:
 *   K codes  8 d bytes: token t, channel 32 c + 8 j + i at byte
 *            t d/2 + 4 (j d/32 + c) + i/2
 *   V codes  8 d bytes: token 8 f + 2 j + e, channel 32 c + 4 r + i at byte
 *            4 ((32 f + 4 r + j) d/32 + c) + 2 e + i/2
 *   K pairs  [16][d / group] of (s, m), then V pairs likewise.
 * These orders are those in which a warp's matrix fragments take them. A byte
 * never holds two tokens, so tokens are written without reading the others.
 *
 * Supported: head_dim 64 or 128; H / Hk in 1..8; page_size 16; bf16 or fp16
 * rows; group 32, 64 or 128, at most head_dim. Others: POD_EUNSUPPORTED.
 *
 * Memory: every pointer is DEVICE memory on the device of the call, the
 * lengths too (int32): nothing is copied from the host, so a captured call
 * that is replayed takes the lengths, tables and rows that its buffers hold
 * then. Rows are 16-byte aligned and strides are in elements, multiples of 8;
 * the channels of a row are adjacent. Outputs may not overlap inputs, except
 * where said. Calls are asynchronous on the given stream (NULL: the legacy
 * default stream), allocate nothing and never synchronise. Host-detectable
 * errors return a negative pod_status (pod_attn.h) before anything is
 * enqueued. What only the device can see is bounded there: no call reads or
 * writes outside the pool, the table or the rows it was given.
 */
#ifndef POD_KV4_H
#define POD_KV4_H

#include "pod_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { POD_DTYPE_BF16 = 0, POD_DTYPE_FP16 = 1 } pod_dtype;

typedef struct pod_kv4_ctx pod_kv4_ctx; /* opaque, library-owned */

typedef struct {
  int num_qo_heads;    /* H (decode only)                                  */
  int num_kv_heads;    /* Hk <= 512; H % Hk == 0                           */
  int head_dim;        /* d: 64 or 128                                     */
  int group_size;      /* channels that share a pair (s, m)                */
  int dtype;           /* pod_dtype of Q, K, V, O rows                     */
  int page_size;       /* 16                                               */
  int max_decode_reqs; /* cap on decodes per call, 1 .. 4096               */
  int device;          /* CUDA device ordinal the context lives on         */
  unsigned flags;      /* 0; POD_FLAG_TEST_FORCE_TIMEOUT (test only): in the
                          context's first pod_kv4_decode warp w of each CTA
                          leaves out the copy of its block 4 w (its last one,
                          if it has fewer), waits for it about 1 ms and gives
                          up                                               */
} pod_kv4_config;

/* Rows of K and V for some requests: the arguments of pod_kv4_write and
 * pod_kv4_read. Row i belongs to the request r with cu_rows[r] <= i <
 * cu_rows[r + 1] and is the token at position start[r] + i - cu_rows[r]. */
typedef struct {
  int num_reqs;             /* entries of start, rows of block_table          */
  int num_rows;             /* rows of k and v; those outside
                               cu_rows[0] .. cu_rows[num_reqs] are left alone */
  const int* cu_rows;       /* device int32 [num_reqs + 1], non-decreasing    */
  const int* start;         /* device int32 [num_reqs]                        */
  void* k;                  /* device [num_rows, Hk, d], read by write and    */
  void* v;                  /*   written by read                              */
  long long k_row_stride, k_head_stride; /* elements                          */
  long long v_row_stride, v_head_stride;
  void* pool;               /* device bytes [pool_blocks, Hk, record], 16-byte aligned */
  long long pool_blocks;
  const int* block_table;   /* device int32 [num_reqs, block_table_stride]    */
  int block_table_stride;
} pod_kv4_rows_args;

/* Decode requests of one call (request r owns Q/O row r). */
typedef struct {
  int num_reqs;             /* 0 .. max_decode_reqs                           */
  const int* ctx_lens;      /* device int32 [num_reqs]; 0: an empty context   */
  const void* q;            /* device [num_reqs, H, d]                        */
  void* o;                  /* device [num_reqs, H, d] (written)              */
  float* lse;               /* device fp32 [num_reqs, H] (written)            */
  const void* pool;         /* device bytes [pool_blocks, Hk, record]         */
  long long pool_blocks;
  const int* block_table;   /* device int32 [num_reqs, block_table_stride]    */
  int block_table_stride;
} pod_kv4_decode_args;

typedef struct {
  int num_qo_heads, num_kv_heads; /* H, Hk: any counts, 0 leaves that side out */
  int head_dim;             /* d: 64 or 128                                   */
  int rot_dim;              /* rotated channels, the first ones: a multiple
                               of 16, 16 .. head_dim                          */
  int interleaved;          /* 0: channel i turns with i + rot_dim / 2,
                               1: channel 2 i with 2 i + 1                    */
  int dtype;                /* pod_dtype of the rows and weights              */
  int device;
  int num_rows;
  const void* q;            /* device [num_rows, H, d]                        */
  const void* k;            /* device [num_rows, Hk, d]                       */
  void* q_out;              /* written; may be q (k) itself with its strides  */
  void* k_out;
  long long q_row_stride, q_head_stride, k_row_stride, k_head_stride;
  long long q_out_row_stride, q_out_head_stride, k_out_row_stride, k_out_head_stride;
  const void* q_weight;     /* device [d], or NULL: no norm, only the rotation */
  const void* k_weight;
  float eps;                /* added to the mean square, >= 0                 */
  const int* positions;     /* device int32 [num_rows]                        */
  const float* cos_sin;     /* device fp32 [max_position, rot_dim]: the cosines
                               of a position, then its sines                  */
  long long max_position;
} pod_qk_args;

/* y = x / sqrt(mean(x^2) + eps) * weight over the d channels of each head,
 * then each pair (a, b) of rotated channels becomes (a cos - b sin,
 * a sin + b cos), in fp32 with one rounding at the end (a head whose mean
 * square passes fp32 becomes 0). A row whose position
 * is negative is padding: neither read nor written. One at max_position or
 * beyond has no angle: its outputs are NaN.
 * Returns POD_OK, POD_EINVAL, POD_EUNSUPPORTED, POD_ECAPACITY or POD_ECUDA. */
POD_API int pod_qk_norm_rope(const pod_qk_args* args, void* stream);

/* Bytes of one (page, KV head) record, 16 d + 128 d / group_size, or a
 * negative pod_status. */
POD_API int pod_kv4_record_bytes(int head_dim, int group_size);

/* Validates cfg and allocates the workspace of pod_kv4_decode on cfg->device.
 * Returns POD_OK, POD_EINVAL, POD_EUNSUPPORTED, POD_ECAPACITY, POD_ENOMEM or
 * POD_ECUDA. */
POD_API int pod_kv4_create(pod_kv4_ctx** out, const pod_kv4_config* cfg);

/* Quantises each row into its place in the cache. Other tokens of the pages
 * it writes to are left as they are. A row whose position lies outside its
 * table row (or below 0), or whose page id lies outside the pool, is not
 * written. The rows of one call have to go to distinct places: where two
 * requests name the same page and offset, that token's contents are a mixture
 * of the two. Calls on one context may overlap (no workspace is used). */
POD_API int pod_kv4_write(pod_kv4_ctx* ctx, const pod_kv4_rows_args* args, void* stream);

/* Writes n * s + m of each row's token, computed in fp32 and rounded once, to
 * k and v. A row that has no place in the cache (as above) becomes NaN. Calls
 * on one context may overlap (no workspace is used). */
POD_API int pod_kv4_read(pod_kv4_ctx* ctx, const pod_kv4_rows_args* args, void* stream);

/* O[r, h] = softmax(q K^T / sqrt(d)) V over the tokens 0 .. ctx_lens[r] - 1
 * as the cache holds them, LSE as in pod_attn.h. Lengths are cut to
 * 0 .. 16 block_table_stride. An empty context gives O = 0 and
 * LSE = -infinity. Scores may be as large as fp32 holds. A request with a page
 * id outside the pool gets O = LSE = NaN, and so do the rows of a device-side
 * wait that ran out (after about a second), which pod_kv4_status then reports.
 * What the cache holds behind a length is never used, whatever its bits.
 * The context's workspace serves one call at a time: calls on one context,
 * replays of captured ones included, must not overlap. */
POD_API int pod_kv4_decode(pod_kv4_ctx* ctx, const pod_kv4_decode_args* args, void* stream);

/* Synchronises `stream`, then returns and clears the sticky device status
 * (POD_OK, or POD_ETIMEOUT after a wait of pod_kv4_decode ran out), or
 * POD_ECUDA if the synchronisation failed. */
POD_API int pod_kv4_status(pod_kv4_ctx* ctx, void* stream);

/* Synchronises the device, reads the sticky status, frees everything. Returns
 * that status (POD_OK or POD_ETIMEOUT) or POD_ECUDA. NULL is a no-op. */
POD_API int pod_kv4_destroy(pod_kv4_ctx* ctx);

#ifdef __cplusplus
}
#endif
#endif /* POD_KV4_H */
