/*
 * hisparse_pages.h -- the resident pages of hisparse_swap_in_resident, kept on
 * the GPU: block tables and slot maps from request lengths, KV rows normalised
 * and stored at those slots, and attention of a whole batch over a prefix that
 * its requests share.
 *
 * The resident tier is a caller's pool of rows in pages of block_size rows:
 * row n of the pool is row n % block_size of page n / block_size.
 * hisparse_page_tables hands out pages as requests grow and takes them back,
 * and names the slot (pool row) of each of a step's new tokens;
 * hisparse_norm_rows writes the tokens' rows there; hisparse_swap_in_resident
 * reads the tables; hisparse_attend reads the rows that a swap-in has flagged;
 * and hisparse_attend_prefix attends over the pages of a prefix that all
 * requests have, once for all of them, and joins that with what hisparse_attend
 * gave for each request's own rows.
 *
 * Conventions (return codes, streams, pointers, graph capture) are those of
 * hisparse.h.  The calls here take no handle and work on the device current at
 * the call.
 *
 * Row formats, by their bytes: 512 latent values, then 64 rope values of the
 * model's 16-bit type.
 *   HISPARSE_ROW4_BYTES   416   4-bit rows (hisparse_rows4.h)
 *   HISPARSE_ROW8_BYTES   656   [0, 512) codes (e4m3), [512, 528) 4 scales
 *                               (float), one per 128 values, [528, 656) rope
 *   HISPARSE_ROW16_BYTES 1152   all values in the model's 16-bit type
 * A latent value of the first two is its code's value times its group's scale.
 */
#ifndef HISPARSE_PAGES_H
#define HISPARSE_PAGES_H

#include <stdint.h>

#include "hisparse_rows4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define HISPARSE_ROW8_BYTES 656
#define HISPARSE_ROW16_BYTES 1152

/* Most tokens of a prefix, and most entries of a block table. */
#define HISPARSE_MAX_PREFIX (1 << 20)
#define HISPARSE_MAX_TABLE_BLOCKS (1 << 20)

/* Arguments of hisparse_page_tables. */
typedef struct hisparse_page_tables_args {
    int32_t num_requests;        /* R >= 1 */
    int32_t max_blocks;          /* entries of a request's table, 1 .. HISPARSE_MAX_TABLE_BLOCKS */
    int32_t block_size;          /* tokens a page, >= 1 */
    int32_t num_shared;          /* entries that belong to a shared prefix, 0 .. max_blocks */
    const int32_t *lens;         /* device-addressable [R] */
    int32_t *tables;             /* device [R] rows of max_blocks, row r at tables + r * tables_stride */
    int64_t tables_stride;
    int32_t *held;               /* device [R] */
    int32_t *free_list;          /* device [free_capacity] */
    int32_t free_capacity;       /* >= 1 */
    int32_t *free_count;         /* device [1] */
    const int32_t *shared;       /* device-addressable [num_shared] (NULL with 0) */
    const int32_t *new_tokens;   /* device-addressable [R], or NULL: no slot map */
    int32_t *offsets;            /* device [R + 1] (with new_tokens) */
    int32_t *slots;              /* device [num_tokens] (with new_tokens) */
    int32_t *positions;          /* device [num_tokens], or NULL */
    int32_t num_tokens;          /* >= 0 */
    int32_t *status;             /* device [R] status words (hisparse_status), or NULL */
} hisparse_page_tables_args;

/*
 * hisparse_page_tables: brings the block tables to the lengths lens, and maps a
 * step's new tokens to slots.
 * A request's table names its pages in order; held[r] entries of it are in use,
 * the others are -1.  Its first num_shared entries belong to the shared prefix
 * (the pages that `shared` names: never taken from the free list, never put
 * there).  free_list[0 .. free_count) are the free pages, the last the next to
 * be taken.
 *  1. A request needs ceil(lens[r] / block_size) entries; with lens[r] < 0 it is
 *     left as it is.  Entries beyond that become -1, and their pages (the
 *     shared ones apart) go to the end of the free list, so that they are taken
 *     again in the order of requests and entries.
 *  2. In the order of the requests, those that need more get it from the end of
 *     the free list, as long as there is enough for a request's whole growth and
 *     that of all before it; the others are left as they are, with status
 *     CAPACITY.
 *  3. new_tokens[r] tokens of request r are new, the last of its lens[r].
 *     offsets[r] is the sum of new_tokens before r (saturated), offsets[R] of all.  Token
 *     i of request r has place offsets[r] + i: positions there is its position
 *     p = lens[r] - new_tokens[r] + i, slots its pool row tables[r][p /
 *     block_size] * block_size + p % block_size.  Both are -1 for the tokens of
 *     requests that are left as they are, of entries that are negative, and at
 *     all places behind the last token.
 * Held entries have to be pages (or shared ones) and each page held or free once.
 * A call with other lengths followed by one with the old ones puts the tables and
 * the list's free pages back as they were (unless a request went without).
 * Data errors, by status: BAD_SEQ_LEN (lens[r] beyond max_blocks pages), BAD_INDEX
 * (held[r] outside [0, max_blocks]): the request is left as it is; BAD_POSITION
 * (new_tokens[r] negative, which counts as 0, or above lens[r]: its tokens get
 * -1); CAPACITY (above, or tokens at or past num_tokens, which are dropped);
 * BAD_RESIDENT (a page whose rows reach HISPARSE_RESIDENT_FLAG: its tokens get -1).
 * A free_count outside [0, free_capacity] is taken as the nearest in it, and pages
 * that the list has no room for are dropped.
 * One launch, or two with many tokens; capturable.  lens, new_tokens and shared
 * may not overlap what the call writes.
 * Errors: INVALID_ARG, UNSUPPORTED (R above HISPARSE_MAX_REQUESTS, max_blocks above
 * its limit, R * max_blocks above 2^31 - 1, block_size or num_tokens above
 * HISPARSE_RESIDENT_FLAG), CUDA.
 */
int hisparse_page_tables(const hisparse_page_tables_args *args, void *stream);

/*
 * hisparse_norm_rows: rows[slots[i]] <- values[i], its latent part normalised
 * and stored in the rows' format, for i < n.
 *   values      device-addressable [n][576] of `dtype`, row i at values + i *
 *               value_stride elements (>= 576, a multiple of 8)
 *   weight      device-addressable [512] of `dtype`, or NULL: no norm, the
 *               values are stored as they are
 *   eps         >= 0
 *   rows        device-addressable [num_rows], row s at rows + s * row_stride
 *               bytes (>= row_bytes, a multiple of 16); pinned host rows are
 *               written over the host link directly
 *   row_bytes   the format
 *   slots       device-addressable int32 [n], or NULL: slot i is i.  A value
 *               whose slot is negative or not below num_rows is not stored.
 *               Of two values with one slot, either's bytes may stand in any
 *               part of the row.
 * With a weight, y = x / sqrt(mean of the 512 x^2 + eps) * weight, not rounded
 * before it is stored (a mean above what 32 bits hold gives 0; one that is 0 in them,
 * with eps 0, NaN); else y = x.  Codes and scales are those of y's exact value, which
 * counts as on a border between two if it is nearer to it than 2^-42 of itself, where
 * the mean is between 2^-100 and 2^100 and the products x * weight are 0 or between
 * 2^-126 and 3.4e38.  (Those that are not are taken as 32 bits have them: bf16's
 * smallest lose bits, its largest are infinite.)  Formats:
 *   1152  y, in 32 bits, rounded to `dtype`
 *    656  group scale: the least power of two, 2^-126 at least, that brings the
 *         group's largest magnitude to 448 or less (infinities: 2^120; NaN: NaN).
 *         A power of two loses nothing to any other scale but at the smallest
 *         codes, and its products with codes are exact in bf16 (and, within its
 *         range, in f16).  Code: the e4m3 value nearest to y / scale, ties to even.
 *    416  as hisparse_pack_rows
 * Rope values are stored as they are.
 * One launch, capturable.  Errors: as hisparse_pack_rows; also INVALID_ARG
 * (row_bytes, num_rows < 0, eps negative or NaN, num_rows < n without slots).
 */
int hisparse_norm_rows(const void *values, int64_t value_stride, int32_t dtype, int64_t n,
                       const void *weight, float eps, void *rows, int64_t row_stride,
                       int32_t row_bytes, int64_t num_rows, const int32_t *slots, void *stream);

/*
 * hisparse_gather_rows: values[i] <- what rows[slots[i]] stands for, each value
 * rounded to `dtype` once (exact but for 656-byte rows whose scales are no powers
 * of two, and beyond f16's range).  Values whose slot is negative or not below
 * num_rows are left as they are.  Arguments and errors as hisparse_norm_rows.
 */
int hisparse_gather_rows(const void *rows, int64_t row_stride, int32_t row_bytes, int64_t num_rows,
                         const int32_t *slots, int64_t n, void *values, int64_t value_stride,
                         int32_t dtype, void *stream);

/* Arguments of hisparse_attend_prefix.  Strides as in hisparse_attend_args. */
typedef struct hisparse_attend_prefix_args {
    int32_t num_requests;          /* R >= 1 */
    int32_t num_heads;             /* H, 1 .. HISPARSE_MAX_HEADS */
    int32_t dtype;                 /* HISPARSE_BF16 or HISPARSE_F16 */
    int32_t row_bytes;             /* the rows' format */
    const void *q;                 /* device [R][H][576]: 512 latent, 64 rope values */
    int64_t q_request_stride;
    int64_t q_head_stride;
    const void *rows;              /* device: the pool, row s at rows + s * row_stride */
    int64_t row_stride;            /* bytes */
    int64_t num_rows;              /* rows there */
    const int32_t *table;          /* device-addressable [ceil(prefix_len / block_size)] */
    int32_t block_size;            /* tokens a page, >= 1 */
    int32_t prefix_len;            /* tokens, 0 .. HISPARSE_MAX_PREFIX */
    float scale;                   /* of the scores, before the softmax */
    const void *part;              /* device [R][H][512] of `dtype`, or NULL */
    int64_t part_request_stride;
    int64_t part_head_stride;
    const float *part_lse;         /* device [R][H] (with part) */
    void *out;                     /* device [R][H][512] of `dtype` */
    int64_t out_request_stride;
    int64_t out_head_stride;
    float *lse;                    /* device [R][H], or NULL */
    int32_t *status;               /* device [R] status words (hisparse_status), or NULL */
    void *workspace;               /* device, 16-byte aligned */
    int64_t workspace_bytes;       /* at least what hisparse_attend_prefix_workspace says */
} hisparse_attend_prefix_args;

/*
 * hisparse_attend_prefix: one decode step's attention of all requests over the
 * prefix_len tokens whose pages `table` names: token t is pool row table[t /
 * block_size] * block_size + t % block_size.  A negative entry names nothing:
 * its tokens are left out (below -1 with status BAD_RESIDENT for every request),
 * and so are tokens whose row is not below num_rows (BAD_RESIDENT too).  For
 * every request r and head h, over the other tokens i:
 *   s[i]      = scale * (q[r][h] . row i)            (576 values)
 *   l         = sum_i exp(s[i]) + exp(part_lse[r][h])
 *   out[r][h] = (sum_i exp(s[i]) latent i + exp(part_lse[r][h]) part[r][h]) / l
 *   lse[r][h] = ln l
 * without the terms of `part` if that is NULL.  part and part_lse may be out and
 * lse themselves: hisparse_attend over a request's own rows, then this call on
 * its results (they may not overlap in any other way).  Where part_lse is -inf,
 * part's values are not looked at.  If there is nothing at all, out = 0 and lse =
 * -inf.
 * Products accumulate in 32 bits (cut off, not rounded, every 16 rows: by a step of
 * 2^-23 at most, 0.8 % in all where 2^20 rows weigh alike).  Latent values are used
 * in `dtype`: exact but as hisparse_gather_rows says.  Probabilities enter the second
 * product in `dtype`, relative to a running maximum (f16: those below 2^-32 of the
 * largest are 0); everything else of the softmax is 32-bit; out is rounded once.
 * Results repeat bit for bit.
 * scale may be any number as long as the scores stay below 2.3e38 (beyond, NaN); in
 * bf16 its power of two is multiplied into the queries, which loses bits of values that
 * come below 2^-126 by it.  A NaN or infinite scale gives NaN wherever a token is named.
 * A bounded wait of the kernel's that runs out (not expected) leaves status
 * ATTEND_TIMEOUT with every request; with status NULL neither that nor
 * BAD_RESIDENT leaves a trace.
 * One to three launches, capturable.  Errors: INVALID_ARG, UNSUPPORTED (R, H or
 * prefix_len beyond the limits), ALIGNMENT (q, rows, part, out or workspace not
 * 16-byte aligned), CAPACITY (workspace too small), CUDA.
 */
int hisparse_attend_prefix(const hisparse_attend_prefix_args *args, void *stream);

/*
 * hisparse_attend_prefix_workspace: *bytes <- the workspace of
 * hisparse_attend_prefix for these sizes.  Its contents need
 * not survive between calls; calls that may overlap on the GPU need a workspace
 * each.  Errors: INVALID_ARG, UNSUPPORTED.
 */
int hisparse_attend_prefix_workspace(int32_t num_requests, int32_t num_heads, int32_t prefix_len,
                                     int64_t *bytes);

#ifdef __cplusplus
}
#endif
#endif /* HISPARSE_PAGES_H */
