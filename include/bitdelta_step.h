/*
 * bitdelta_step.h -- what a serving step needs between the linears of
 * bitdelta.h: the RMS norm that makes a linear's bf16 x out of the previous
 * linear's result, the paged key-value cache, and the attention of one new
 * token over it.
 *
 * "Serving architecture" of the post (see bitdelta.h) keeps one base and many
 * deltas on a GPU, which leaves little of its memory for keys and values:
 * with a 70B base and 14 variants resident (257 of 288 GB) the cache decides
 * how many requests fit, so its rows can be held in 8 bits.
 *
 * The conventions of bitdelta.h hold (device pointers, asynchronous calls on
 * `stream`, caller-owned buffers, argument errors before anything is
 * enqueued, BD_ERR_DEVICE off gfx950), with these additions:
 *
 * - Types are named per argument by a bd_type; another value is BD_ERR_MODE.
 * - e4m3 groups.  A group of values is held as OCP e4m3 codes and one scale
 *   byte: with a the largest magnitude among the group's finite values, e is
 *   the smallest whole number, at least -111, for which a <= 448 * 2^e; the
 *   byte is e + 127 and the code of x is x / 2^e rounded to e4m3 (nearest,
 *   ties to even).  A value that is not finite gets the NaN code.  The scale
 *   is a power of two because an e4m3 code's relative step does not depend
 *   on it: the division and the read-back are exact, and 448 is never passed.
 *   Code times scale is exact in bf16 (a value so large that it rounds to
 *   2^128 reads as infinity, as it does when rounded to bf16).
 * - Ids, slots, pages and lengths live on the device and cannot be checked on
 *   the host: each call says what it does with one out of range.  None makes
 *   it touch memory outside the arguments.
 */
#ifndef BITDELTA_STEP_H
#define BITDELTA_STEP_H

#include "bitdelta.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum bd_type {
    BD_BF16 = 0,
    BD_FP32 = 1,
    BD_E4M3 = 2
} bd_type;

/* ---------------------------------------------------------------------------
 * RMS norm, with the residual's addition before it.
 *
 *   h = x + residual  (fp32; without a residual h = x)
 *   residual_out = h rounded to residual_type, and h stands for that value
 *   y = h / sqrt(mean(h^2) + eps) * gain[variant]
 *
 *   x            [M, d], x_type BD_BF16 or BD_FP32 (the linears give either).
 *   residual     [M, d], residual_type BD_BF16 or BD_FP32; NULL for none.
 *   residual_out [M, d], written; may be `residual` itself, and only that
 *                (no other overlap).  NULL exactly where residual is.
 *   gain         [num_gains, d], gain_type BD_BF16 or BD_FP32.
 *   variant_ids  [M] int32; token m uses gain variant_ids[m] (each variant
 *                keeps its own norm gains, which no delta holds).  NULL: gain
 *                0 for every token.  An id outside [0, num_gains) gives a row
 *                of NaN (NaN codes, scale byte 127); residual_out is written.
 *   out          [M, d]: BD_BF16 (y rounded once), or BD_E4M3 codes.
 *   scales       [M, ceil(d / 32)] uint8 for BD_E4M3: groups of 32 columns,
 *                the last one of the rest.  NULL for BD_BF16.
 * d: a multiple of 8, 8 .. 65536.  eps >= 0.  x, residual, residual_out,
 * gain, out: 16-byte aligned (out: 8 for BD_E4M3).  M <= 2^31 - 1; M == 0 is
 * a no-op.
 * fp32 throughout for a bf16 result (a row whose squares leave fp32's range is
 * scaled by a power of two first, so h may be of any size); for codes the sum,
 * root and products are 64-bit and y is rounded once, to its code (a finite y
 * past the largest fp32 number counts as that).  Fixed order: the same inputs
 * give bitwise the same outputs.
 * Returns BD_OK, BD_ERR_NULL, _SHAPE, _ALIGN, _MODE, _HIP, _DEVICE.
 * ------------------------------------------------------------------------- */
bd_status bd_rms_norm(const void* x, int32_t x_type, const void* residual, void* residual_out,
                      int32_t residual_type, const void* gain, int32_t gain_type, int32_t num_gains,
                      const int32_t* variant_ids, float eps, void* out, int32_t out_type, uint8_t* scales,
                      int64_t M, int64_t d, void* stream);

/* ---------------------------------------------------------------------------
 * The paged key-value cache: two arrays of pages, each with `page_size`
 * tokens of `num_heads` rows of `head_dim` values.  Token `slot` is place
 * slot % page_size of page slot / page_size; its row of head h starts at
 * element page * page_stride + h * head_stride + place * token_stride, in
 * `k` and in `v` alike.
 *
 *   type       BD_BF16 or BD_E4M3 (one group per row).
 *   k_scales, v_scales   BD_E4M3: [num_pages, num_heads, page_size] uint8,
 *              contiguous, 8-byte aligned; NULL for BD_BF16.
 *   num_pages  >= 1, num_pages * page_size <= 2^31 - 1.
 *   page_size  a multiple of 8, 8 .. 4096.
 *   num_heads  1 .. 65535.
 *   head_dim   a multiple of 16, 16 .. 256.
 *   strides    in elements, >= 0, multiples of 16 bytes and below 2^36 bytes;
 *              distinct rows must not overlap.  k, v: 16-byte aligned.
 * Rows of k, rows of v, k_scales and v_scales lie apart from each other (k's
 * and v's may lie in the gaps of each other's strides).
 * The struct is read during the call only.
 * ------------------------------------------------------------------------- */
typedef struct bd_kv {
    void* k;
    void* v;
    uint8_t* k_scales;
    uint8_t* v_scales;
    int32_t type;
    int32_t num_heads;
    int32_t head_dim;
    int32_t page_size;
    int64_t num_pages;
    int64_t page_stride;
    int64_t head_stride;
    int64_t token_stride;
} bd_kv;

/* Writes the keys and values of T tokens into their slots.
 *
 *   k, v     T tokens of num_heads rows of head_dim values, in_type BD_BF16
 *            or BD_FP32, 16-byte aligned: token t's row of head h starts at
 *            element t * k_strides[0] + h * k_strides[1] (v likewise).  The
 *            strides are HOST arrays of two, multiples of 16 bytes.  These rows
 *            and `slots` lie apart from the cache's rows and scale bytes (the
 *            gaps of its strides are free); to move rows within a cache, copy
 *            them out first.
 *   slots    [T] int32.  A slot below 0 or past the last page: that token is
 *            not written.  A slot named by several tokens holds the last of
 *            them afterwards.
 * A BD_BF16 cache rounds once (nearest even); a BD_E4M3 cache holds each row
 * as one group.  Every other slot stays as it was.  T <= 2^28; T == 0 is a
 * no-op.
 * Returns BD_OK, BD_ERR_NULL, _SHAPE, _ALIGN, _MODE, _HIP, _DEVICE. */
bd_status bd_kv_write(const bd_kv* kv, const void* k, const int64_t* k_strides, const void* v,
                      const int64_t* v_strides, int32_t in_type, const int32_t* slots, int64_t T, void* stream);

/* Reads rows back: k_out, v_out [T, num_heads, head_dim] bf16, 16-byte
 * aligned, apart from each other, the slots and the cache's rows and scale
 * bytes; the exact value of every held row.  A slot below 0 gives zeros (a
 * padding token), one past the last page NaN.  T <= 2^31 - 1; T == 0 is a
 * no-op.
 * Returns BD_OK, BD_ERR_NULL, _SHAPE, _ALIGN, _MODE, _HIP, _DEVICE. */
bd_status bd_kv_read(const bd_kv* kv, const int32_t* slots, int64_t T, uint16_t* k_out, uint16_t* v_out,
                     void* stream);

/* ---------------------------------------------------------------------------
 * Attention of one new token per sequence over the cache.
 *
 *   out[b, i] = sum_j softmax_j(scale * q[b, i] . k_j) v_j,   j < lengths[b]
 *
 * where k_j, v_j are the rows of head i / (num_q_heads / num_heads) of the
 * sequence's token j, which is in page page_table[b][j / page_size].
 *
 *   q           B tokens of num_q_heads rows of head_dim values, q_type
 *               BD_BF16 or BD_FP32, 16-byte aligned: row (b, i) starts at
 *               element b * q_strides[0] + i * q_strides[1] (HOST array of
 *               two, multiples of 16 bytes).  num_q_heads is a multiple of
 *               num_heads, at most 65535.
 *   page_table  [B, max_pages] int32, rows table_stride elements apart.
 *               max_pages * page_size <= 2^24; with R = B * num_heads *
 *               ceil(num_q_heads / num_heads / 16) rows of
 *               U = ceil(max_pages * page_size / 128) units, R <= 2^23 and
 *               R * (U + 4) <= 2^30.
 *   lengths     [B] int32: tokens to attend to, the new one among them (its
 *               row has been written by then).  0 or less: the sequence's
 *               rows of out are zeros, of lse -infinity.  Only the pages that
 *               hold these tokens are looked up, and what lies behind the
 *               last token in its page does not matter, NaN included.
 *               A length over max_pages * page_size, or a looked-up page
 *               outside [0, num_pages), gives rows of NaN.
 *   scale       multiplies the scores q . k; of any sign, 2^60 at most in
 *               magnitude.  Scores may be of any size before and after it:
 *               only a q . k itself past fp32's range counts as infinite,
 *               and an fp32 query value that rounds to infinity in bf16.
 *   out         [B, num_q_heads, head_dim] bf16, 16-byte aligned.
 *   lse         [B, num_q_heads] fp32, the natural logarithm of
 *               sum_j exp(scale * q . k_j); NULL if not wanted.  out and lse
 *               lie apart from each other and from all that is read.
 *   workspace   device scratch of at least bd_attend_workspace_bytes(...)
 *               bytes, 16-byte aligned; may be NULL when that is 0.  The
 *               tokens of all sequences are split evenly over the GPU; the
 *               fp32 partial results of a sequence that several workgroups
 *               share live there until they are joined, in a fixed order.
 *               Its contents on entry do not matter.  Where the table holds
 *               few tokens for each sequence nothing is split, and it is 0.
 * Scores, the running maximum and sum and the output sums are fp32; fp32
 * queries enter the matrix products as three bf16 terms, which hold all of
 * their bits, the softmax weights as two, 16 bits (but where a row of the
 * sequence itself holds infinities: what they reach is summed with one term
 * each, as further ones would make NaN of them).  The same inputs and
 * batch give bitwise the same outputs.  B == 0 is a no-op.
 * Returns BD_OK, BD_ERR_NULL, _SHAPE, _ALIGN, _MODE, _WORKSPACE, _HIP,
 * _DEVICE.
 * ------------------------------------------------------------------------- */
size_t bd_attend_workspace_bytes(int64_t B, int64_t num_q_heads, int64_t num_heads, int64_t head_dim,
                                 int64_t page_size, int64_t max_pages);
bd_status bd_attend(const bd_kv* kv, const void* q, int32_t q_type, const int64_t* q_strides,
                    int32_t num_q_heads, const int32_t* page_table, int64_t table_stride, int64_t max_pages,
                    const int32_t* lengths, int64_t B, float scale, uint16_t* out, float* lse,
                    void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BITDELTA_STEP_H */
