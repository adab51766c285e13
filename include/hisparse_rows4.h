/*
 * hisparse_rows4.h -- KV rows held in 4 bits: packing, attention over them by
 * slot id, and eviction of the hot rows with the least attention weight.
 *
 * These calls sit around the swap-in of hisparse.h.  A handle created with
 * row_bytes = HISPARSE_ROW4_BYTES stores packed rows in its pinned pool and
 * hot buffers (hisparse_pack_rows makes them, for the prefix and for each
 * step's backup); hisparse_attend reads them by the slot ids that a swap-in
 * wrote and adds each token's attention weight to an accumulator; and
 * hisparse_evict frees the hot rows of the least accumulated weight, which
 * the next swap-in's misses then fill first.
 *
 * Conventions (return codes, streams, pointers, graph capture) are those of
 * hisparse.h.  The calls here that take no handle work on the device current
 * at the call.
 *
 * A 4-bit row, HISPARSE_ROW4_BYTES bytes:
 *   [  0, 256)  512 latent values as 4-bit codes (e2m1: sign, two exponent
 *               bits, one mantissa bit; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4,
 *               6); value 2b in the low half of byte b, 2b + 1 in the high
 *   [256, 288)  32 scales (e4m3), one per 16 latent values
 *   [288, 416)  64 rope values of the model's 16-bit type
 * A latent value is its code's value times its group's scale: at most six
 * significant bits, so it is exact in bf16 and in f16.
 */
#ifndef HISPARSE_ROWS4_H
#define HISPARSE_ROWS4_H

#include <stdint.h>

#include "hisparse.h"

#ifdef __cplusplus
extern "C" {
#endif

#define HISPARSE_ROW4_LATENT 512
#define HISPARSE_ROW4_ROPE 64
#define HISPARSE_ROW4_VALUES 576   /* latent, then rope */
#define HISPARSE_ROW4_BYTES 416

/* The 16-bit type of values, queries and outputs. */
#define HISPARSE_BF16 0
#define HISPARSE_F16 1

/* Status code (see hisparse_status): an attention kernel's own bounded wait
 * ran out (not expected; the request's outputs and the weights added by the
 * call are not valid). */
#define HISPARSE_STATUS_ATTEND_TIMEOUT 9

/* Most rows of one hisparse_pack_rows or hisparse_unpack_rows. */
#define HISPARSE_MAX_PACKED_ROWS (4 * (int64_t)0x7FFFFFFF)

/* Limits of hisparse_attend; top_k is at most HISPARSE_MAX_TOP_K. */
#define HISPARSE_MAX_HEADS 1024

/*
 * hisparse_pack_rows: rows[i] <- values[i] in 4 bits, i < n.
 *   values        device-addressable [n][576] of `dtype`, row i at
 *                 values + i * value_stride elements (>= 576, a multiple of 8)
 *   rows          device-addressable, row i at rows + i * row_stride bytes
 *                 (>= 416, a multiple of 16); pinned host rows are written
 *                 over the host link directly
 * Group scale: the e4m3 value nearest to (largest magnitude of the 16) / 6,
 * at most 448, ties to even.  Code: the e2m1 value nearest to value / scale,
 * ties to the even code, at most 6 in magnitude; 0 where the scale is 0.
 * Infinities clip to 6 * 448; a NaN makes its group's scale NaN, and with it
 * the group's values.  The sign bit of a code is the value's, also at 0.
 * Errors: INVALID_ARG (null, n < 0, a short or odd stride, dtype), UNSUPPORTED
 * (n > HISPARSE_MAX_PACKED_ROWS), ALIGNMENT (pointers not 16-byte aligned),
 * CUDA.  n = 0 does nothing.
 */
int hisparse_pack_rows(const void *values, int64_t value_stride, int32_t dtype, int64_t n,
                       void *rows, int64_t row_stride, void *stream);

/*
 * hisparse_unpack_rows: values[i] <- what rows[i] stands for (exact in both
 * types), for readers of the hot buffer that want 16-bit rows.  Arguments
 * and errors as hisparse_pack_rows.
 */
int hisparse_unpack_rows(const void *rows, int64_t row_stride, int64_t n, void *values,
                         int64_t value_stride, int32_t dtype, void *stream);

/*
 * Arguments of hisparse_attend.  Strides of q and out are in elements (of
 * `dtype`), multiples of 8; row strides are in bytes, multiples of 16.  The
 * request and head strides of a single request or head are not looked at;
 * otherwise those of out are at least 512 apart.
 */
typedef struct hisparse_attend_args {
    int32_t num_requests;          /* R >= 1 */
    int32_t num_heads;             /* H, 1 .. HISPARSE_MAX_HEADS */
    int32_t top_k;                 /* k, 1 .. HISPARSE_MAX_TOP_K */
    int32_t dtype;                 /* HISPARSE_BF16 or HISPARSE_F16 */
    const void *q;                 /* device [R][H][576]: 512 latent, 64 rope values */
    int64_t q_request_stride;
    int64_t q_head_stride;
    const void *rows;              /* device: row s of request r at
                                      rows + r * request_stride + s * row_stride */
    int64_t row_stride;
    int64_t request_stride;
    int32_t rows_per_request;      /* D: hot slots are [0, D) */
    float scale;                   /* of the scores, before the softmax */
    const int32_t *slot_ids;       /* device-addressable [R][k], row r at slot_ids + r * ids_stride */
    int64_t ids_stride;
    const void *resident_rows;     /* device rows that flagged ids name, or NULL */
    int64_t resident_stride;
    int64_t resident_count;        /* rows there (0 with NULL) */
    void *out;                     /* device [R][H][512] of `dtype` */
    int64_t out_request_stride;
    int64_t out_head_stride;
    float *lse;                    /* device [R][H], or NULL */
    float *weights;                /* device accumulators, request r's at
                                      weights + r * weights_stride, or NULL */
    int64_t weights_stride;
    int64_t weights_tokens;        /* accumulators per request, <= weights_stride */
    const int32_t *positions;      /* device-addressable [R][k] token positions
                                      (with weights), row r at + r * positions_stride */
    int64_t positions_stride;
    int32_t *status;               /* device [R] status words (hisparse_status), or NULL */
    void *workspace;               /* device, 16-byte aligned */
    int64_t workspace_bytes;       /* at least what hisparse_attend_workspace says */
} hisparse_attend_args;

/*
 * hisparse_attend: one decode step's sparse attention over 4-bit rows.
 * Request r's rows are those that slot_ids[r] names, as a swap-in wrote it:
 * id < D a hot slot, HISPARSE_RESIDENT_FLAG | n row n of resident_rows, -1
 * nothing.  For every head h, over the named rows i:
 *   s[i]      = scale * (q[r][h] . row i)           (576 values)
 *   out[r][h] = sum_i softmax(s)[i] * latent i      (512 values)
 *   lse[r][h] = ln sum_i exp(s[i])
 *   weights[r][positions[r][i]] += sum over h of softmax(s)[i]
 * A request that names nothing gets out = 0, lse = -inf and no weight.  A
 * row may be named twice (it counts twice).  Products accumulate in 32 bits;
 * probabilities enter the second product as f16 relative to a running
 * maximum (half a step: 2^-11 of a probability, and never less than 2^-25 of
 * that maximum: far smaller ones are dropped from out, not from lse and
 * weights), everything else of the softmax is 32-bit; out is rounded once.
 * Queries are exact down to 2^-22 (rope values in f16: 2^-14) of the largest
 * value of their head, and rounded to 2^-31 (2^-24) of it below.
 * Results do not depend on the batch's other requests' values, and a call
 * repeated on the same inputs gives the same bits if each request's positions
 * are distinct.
 * Ids outside these ranges are skipped and recorded in status: BAD_INDEX for
 * an id below -1 or a slot >= D, BAD_RESIDENT for a flagged id past
 * resident_count, BAD_POSITION for a named row's position outside
 * [0, weights_tokens) (its weight is dropped).  With status NULL
 * neither these nor ATTEND_TIMEOUT leave a trace.
 * Scores of 2^25 and more in magnitude are beyond what the running maximum is kept
 * in: out and lse may then be 0 or NaN.
 * A NaN scale gives NaN wherever a row is named.  One to four launches,
 * capturable.
 * Errors: INVALID_ARG, UNSUPPORTED (H or k beyond the limits), ALIGNMENT
 * (q, rows, resident_rows, out or workspace not 16-byte aligned), CAPACITY
 * (workspace too small), CUDA.
 */
int hisparse_attend(const hisparse_attend_args *args, void *stream);

/*
 * hisparse_attend_workspace: *bytes <- the workspace of hisparse_attend for
 * these sizes (with_weights: weights are asked for).  Its contents need not
 * survive between calls; calls that may overlap on the GPU need a workspace
 * each.  Errors: INVALID_ARG, UNSUPPORTED.
 */
int hisparse_attend_workspace(int32_t num_requests, int32_t num_heads, int32_t top_k,
                              int32_t with_weights, int64_t *bytes);

/*
 * hisparse_evict_select: which cached tokens to give up, by accumulated
 * attention weight.  Nothing is freed.
 *   weights     device [R] rows of float, request r's at weights + r *
 *               weights_stride: one per token position, weights_tokens of
 *               them (<= weights_stride; with 0, weights may be NULL)
 *   slot2tok    device int32 [R][D]: the token in each slot, or -1
 *   seq_lens    device-addressable int32 [R]
 *   keep_recent tokens at the end of each request that are never given up
 *   n           slots to choose per request, 1 <= n <= D
 *   want        device-addressable int32 [R]: as n for each request (clamped
 *               to [0, n]), or NULL: n for all
 *   out_slots   device int32 [R][n]; out_counts device int32 [R]
 * Candidates of request r are the slots whose token t satisfies 0 <= t <
 * seq_lens[r] - keep_recent and t < weights_tokens; a request with
 * seq_lens[r] <= D has none (its buffer holds every token at slot = token).
 * The candidates with the least (weight, slot) are chosen (a NaN weight
 * counts as the largest, -0 as 0) and written in ascending slot order,
 * followed by -1; out_counts is how many there are.
 * Errors: INVALID_ARG, UNSUPPORTED (D above HISPARSE_MAX_DEVICE_BUFFER), CUDA.
 */
int hisparse_evict_select(int32_t num_requests, int32_t rows_per_request, const float *weights,
                          int64_t weights_stride, int64_t weights_tokens, const int32_t *slot2tok,
                          const int32_t *seq_lens, int32_t keep_recent, int32_t n,
                          const int32_t *want, int32_t *out_slots, int32_t *out_counts,
                          void *stream);

/*
 * hisparse_evict: hisparse_evict_select on the hot state of a handle's
 * layer, and free the chosen slots: their tokens are unmapped, their stamps
 * become 0 and they move to the front of the LRU order (which stays sorted
 * by (last_used, slot)), so the next swap-in's misses take them before any
 * other row.  Slots that the last hisparse_set_protected_calls calls
 * selected are no candidates.  The rows stay in the host pool; a freed token
 * that is selected again is a miss.  With layers anchored on `layer` the
 * freed slots are freed in them too (they share its maps).
 *   weights, weights_stride, weights_tokens, seq_lens, keep_recent, n, want
 *                          as above
 *   out_slots, out_counts  as above, or NULL
 * One launch, capturable.  Errors: INVALID_ARG, LAYER, CUDA.
 */
int hisparse_evict(hisparse_t h, int32_t layer, const float *weights, int64_t weights_stride,
                   int64_t weights_tokens, const int32_t *seq_lens, int32_t keep_recent, int32_t n,
                   const int32_t *want, int32_t *out_slots, int32_t *out_counts, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* HISPARSE_ROWS4_H */
