/*
 * bconv_mx4.h -- microscaled 4-bit floating point and layers of experts on AMD
 * Instinct MI355X (gfx950), next to the 4-bit integer operators of bconv_q4.h.
 *
 * C ABI of libbconv.so, continued.  Operators that are used together:
 *
 *   bconv_mx4_quantize   rows to 4-bit floats with one power of two per 32
 *                        values;
 *   bconv_mx4_linear_*   linear layers whose weights and inputs are such
 *                        numbers: one layer, or one for each expert with the
 *                        rows that chose it;
 *   bconv_expert_sort    (token, choice) pairs sorted by expert;
 *   bconv_expert_gather, bconv_expert_combine and their gradients
 *                        tokens' rows into that order, and back with weights.
 *
 * Conventions are those of bconv.h: every call returns a bconv_status_t,
 * argument errors are found on the host before anything is launched,
 * bconv_last_error() has the text; calls are asynchronous on `stream` (a
 * hipStream_t; NULL = default stream), never allocate and never synchronise,
 * so they can be captured in a HIP graph (bconv_mx4_linear_create and _destroy
 * do both and cannot); buffers are the caller's device
 * memory and must stay valid until the stream's work completes.  Calls
 * without a handle run on the current HIP device; a handle's are launched on
 * the device it was created on, to which their buffers and stream belong.
 * Rows may start at any element; row strides are at most 2^30 elements.
 */
#ifndef BCONV_MX4_H
#define BCONV_MX4_H

#include "bconv_q4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Microscaled 4-bit floats
 *
 * A row is cut into blocks of 32 values (the last may be short).  A block has
 * a power of two 2^e, held as the byte e + 127, and a value x of it the 4-bit
 * code nearest to x / 2^e: bit 3 the sign, bits 0..2 the magnitude
 *   0, 0.5, 1, 1.5, 2, 3, 4, 6,
 * ties to the even code, more than 6 to 6.  With m the largest |x| of the block,
 *   e = max(floor(log2 m) - 2, -127)      (-127 for a block of zeros),
 * so that m / 2^e is below 8.  A block that holds a NaN or an infinity has the
 * byte 255, which makes all of it NaN, and codes 0.
 * ------------------------------------------------------------------------ */

/* Quantised rows of `cols` values in device memory, dense: with
 * padded = cols rounded up to a multiple of 256,
 *   codes   [rows][padded / 2]   value 2 i in the low half of byte i,
 *   scales  [rows][padded / 32]  a byte a block.
 * Padding values are 0 (codes 0, bytes 0). */
#define BCONV_MX4_BLOCK 32
#define BCONV_MX4_PAD 256

/* Quantises `rows` rows of `cols` values of `dtype`; row m starts at x + m*ldx
 * (elements, ldx >= cols).  codes (16-byte aligned) and scales (8-byte aligned) receive the
 * quantised rows in the layout above.  `values`, when given, receives what they
 * stand for: dense [rows][cols] of `dtype`, in which every such number is
 * exact.  Results overlap neither x nor each other.  rows == 0 is a no-op;
 * cols is in [1, 2^20]. */
bconv_status_t bconv_mx4_quantize(void *stream, int32_t rows, int32_t cols, int32_t dtype, const void *x, int64_t ldx,
                                  uint8_t *codes, uint8_t *scales, void *values);

/* ------------------------------------------------------------------------
 * Linear layers of microscaled 4-bit floats
 *
 *   y[i][o] = bias[f][o] + sum_k Q(x[r])[k] * W[f][o][k]
 *
 * for row i of the expert f that it belongs to, from input row r; one layer
 * without experts is one expert with all rows, r = i.  Q quantises as above,
 * whatever the number of rows; products are exact, sums are fp32, results are rounded to
 * `dtype` once.  (Sums below the normal fp32 numbers, from blocks whose powers of two
 * multiply to less, lose bits or become 0; sums beyond fp32 become infinite.)
 * ------------------------------------------------------------------------ */

typedef struct bconv_mx4_linear *bconv_mx4_linear_t;

typedef struct {
    int32_t experts;      /* 1 .. 1024 */
    int32_t in_features;  /* 1 .. 2^20 */
    int32_t out_features; /* 1 .. 2^20; experts * in_features * out_features <= 2^38 */
} bconv_mx4_linear_desc_t;

/* Builds layers on the current HIP device from device memory:
 *   codes   uint8 [experts][out_features][ceil(in_features/2)], value 2 i of a
 *           row in the low half of byte i (an unused last half is ignored)
 *   scales  uint8 [experts][out_features][ceil(in_features/32)], e + 127; 255: NaN
 *   bias    float [experts][out_features] or NULL (-> 0)
 * Everything is copied and rearranged by work on `stream`, which the call
 * waits for; the caller keeps its buffers. */
bconv_status_t bconv_mx4_linear_create(const bconv_mx4_linear_desc_t *desc, void *stream, const uint8_t *codes,
                                       const uint8_t *scales, const float *bias, bconv_mx4_linear_t *out);

typedef struct {
    const void *x;           /* input rows, elements of `dtype`: row r at x + r*ldx; or NULL */
    int64_t ldx;             /* >= in_features */
    const uint8_t *codes;    /* with x NULL: input rows as bconv_mx4_quantize lays them out */
    const uint8_t *scales;   /*              (16-byte aligned) */
    void *y;                 /* [rows][out_features], row i at y + i*ldy; overlaps nothing else (y and x may be
                                columns of one buffer: the same stride, no element of both) */
    int64_t ldy;             /* >= out_features */
    int32_t x_rows;          /* input rows; with offsets, x_rows times in_features (rounded up to a
                                multiple of 256) is at most 2^32 */
    int32_t rows;            /* result rows; with offsets at most 2^27 */
    int32_t dtype;           /* of x and y */
    int32_t choices;         /* 0: result row i is of input row i (x_rows == rows); otherwise of
                                order[i] / choices, and x_rows == rows / choices */
    const int32_t *offsets;  /* device [experts + 1]: rows offsets[f] .. offsets[f+1]-1 are expert f's;
                                NULL for one expert: all rows */
    const int32_t *order;    /* device [rows] with choices > 0 (offsets then too), otherwise NULL */
} bconv_mx4_rows_t;

/* Workspace bytes the call needs (0 is possible); host only, looks at pointers
 * only for whether x and offsets are NULL. */
bconv_status_t bconv_mx4_linear_workspace_size(bconv_mx4_linear_t h, const bconv_mx4_rows_t *args, size_t *bytes);

/* y = the formula above.  offsets and order are those of bconv_expert_sort
 * (offsets outside [0, rows] and input rows outside [0, x_rows) count as the
 * nearest inside).  Rows from offsets[experts] on become 0.  rows == 0 is a
 * no-op.  The workspace is 16-byte aligned and overlaps nothing; its contents
 * need not be kept between calls. */
bconv_status_t bconv_mx4_linear_forward(bconv_mx4_linear_t h, void *stream, const bconv_mx4_rows_t *args,
                                        void *workspace, size_t workspace_bytes);

/* Releases the handle's device memory (no queued call may still use it).  NULL is accepted. */
bconv_status_t bconv_mx4_linear_destroy(bconv_mx4_linear_t h);

/* ------------------------------------------------------------------------
 * Tokens to experts and back
 *
 * `choices` experts a token make tokens * choices pairs; pair t * choices + j
 * is choice j of token t.  A pair whose id is not in [0, experts) is dropped.
 * ------------------------------------------------------------------------ */

/* Sorts the pairs by expert, those of an expert in their order.
 *   ids       device, int32 or int64 (id_bytes 4 or 8) [pairs]
 *   offsets   [experts + 1] where each expert's pairs start; the last is the
 *             number of pairs that are not dropped
 *   order     [pairs] the pair at each place; -1 from offsets[experts] on
 *   position  [pairs] the place of each pair; -1 for dropped ones
 * experts is in [1, 1024], pairs in [0, 2^27].  offsets is written for pairs == 0 too. */
bconv_status_t bconv_expert_sort_workspace_size(int32_t pairs, int32_t experts, size_t *bytes);
bconv_status_t bconv_expert_sort(void *stream, int32_t pairs, int32_t experts, int32_t id_bytes, const void *ids,
                                 int32_t *offsets, int32_t *order, int32_t *position, void *workspace,
                                 size_t workspace_bytes);

/* rows[p] = x[t] for each pair's place p = position[t*choices + j]; places whose
 * order entry is negative become 0.  x: [tokens][width] of `dtype`, row t at
 * x + t*ldx; rows: dense [tokens * choices][width].  width is in [1, 2^20],
 * tokens * choices at most 2^27. */
bconv_status_t bconv_expert_gather(void *stream, int32_t tokens, int32_t choices, int32_t width, int32_t dtype,
                                   const void *x, int64_t ldx, const int32_t *order, const int32_t *position, void *rows);

/* y[t] = sum_j weights[t][j] * rows[position[t*choices + j]] over the pairs that
 * are not dropped, summed in fp32 in the order of j; 0 for a token without any.
 * rows: row p at rows + p*ldr; y: dense [tokens][width]; weights: dense
 * [tokens][choices] of `weight_dtype`, or NULL for 1 (the gradient of the
 * gather: dx from the gradient of its rows). */
bconv_status_t bconv_expert_combine(void *stream, int32_t tokens, int32_t choices, int32_t width, int32_t dtype,
                                    const void *rows, int64_t ldr, const int32_t *position, int32_t weight_dtype,
                                    const void *weights, void *y);

/* Gradients of the combination for the gradient dy of y (row t at dy + t*ldd):
 *   d_rows[position[t*choices + j]] = weights[t][j] * dy[t]   (0 at places whose order entry is negative)
 *   d_weights[t][j] = <dy[t], rows[position[t*choices + j]]>  (0 for dropped pairs), summed in fp32
 * d_rows is dense [tokens * choices][width], d_weights dense [tokens][choices]
 * of weight_dtype.  weights NULL counts as 1; d_weights may be NULL, rows too then. */
bconv_status_t bconv_expert_combine_backward(void *stream, int32_t tokens, int32_t choices, int32_t width,
                                             int32_t dtype, const void *dy, int64_t ldd, const void *rows, int64_t ldr,
                                             const int32_t *order, const int32_t *position, int32_t weight_dtype,
                                             const void *weights, void *d_rows, void *d_weights);

#ifdef __cplusplus
}
#endif

#endif /* BCONV_MX4_H */
