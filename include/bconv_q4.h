/*
 * bconv_q4.h -- 4-bit operators of a language model's decoding step on AMD
 * Instinct MI355X (gfx950), next to the binary layers of bconv.h.
 *
 * C ABI of libbconv.so, continued.  Four operators that are used together:
 *
 *   bconv_q4_linear_*   linear layers with 4-bit weights and group scales;
 *   bconv_block_tables  block tables and slot maps of a paged cache, built on
 *                       the GPU from request lengths;
 *   bconv_kv4_append    the write of new keys and values into a paged cache
 *                       held in 4 bits;
 *   bconv_kv4_attention attention over that cache, from one token a request
 *                       to prompts.
 *
 * Conventions are those of bconv.h: every call returns a bconv_status_t,
 * argument errors are found on the host before anything is launched,
 * bconv_last_error() has the text; calls are asynchronous on `stream` (a
 * hipStream_t; NULL = default stream), never allocate and never synchronise,
 * so they can be captured in a HIP graph; buffers are the caller's device
 * memory and must stay valid until the stream's work completes.  Calls
 * without a handle run on the current HIP device; a handle's are launched on
 * the device it was created on, to which their buffers and stream belong.
 */
#ifndef BCONV_Q4_H
#define BCONV_Q4_H

#include "bconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations.  Sums, softmax statistics and scales are
 * fp32 whatever the type; results are rounded to it once. */
typedef enum {
    BCONV_F32 = 0,
    BCONV_F16 = 1,
    BCONV_BF16 = 2
} bconv_dtype_t;

/* ------------------------------------------------------------------------
 * Linear layers with 4-bit weights
 *
 *   y[m][o] = bias[o] + sum_k x[m][k] * scale[o][k / group]
 *                                     * (code[o][k] - zero[o][k / group])
 * ------------------------------------------------------------------------ */

typedef struct bconv_q4_linear *bconv_q4_linear_t;

typedef struct {
    int32_t in_features;  /* 1 .. 2^20 */
    int32_t out_features; /* 1 .. 2^20; in_features * out_features <= 2^34 */
    int32_t group;        /* inputs that share a scale: 32, 64 or 128 (the last group may be short) */
} bconv_q4_linear_desc_t;

/* Builds a layer on the current HIP device.
 *   weight_words  host, uint32 [out_features][ceil(in_features/8)]: input i is
 *                 bits 4*(i%8) .. 4*(i%8)+3 of word i/8; nibbles past
 *                 in_features are ignored
 *   scales        host, IEEE fp16 bits [out_features][ceil(in_features/group)]
 *   zeros         host, uint8 of the same shape, each 0..15, or NULL (-> 8)
 *   bias          host, float [out_features] or NULL (-> 0)
 * Every array is copied and rearranged on the device; the caller keeps its
 * buffers.  Synchronous. */
bconv_status_t bconv_q4_linear_create(const bconv_q4_linear_desc_t *desc, const uint32_t *weight_words,
                                      const uint16_t *scales, const uint8_t *zeros, const float *bias,
                                      bconv_q4_linear_t *out);

/* Workspace bytes a forward call with `rows` rows of `dtype` needs (0 is possible). */
bconv_status_t bconv_q4_linear_workspace_size(bconv_q4_linear_t h, int32_t rows, int32_t dtype, size_t *bytes);

/* y = the formula above for `rows` rows.  x and y hold elements of `dtype`;
 * row m starts at x + m*ldx (ldx >= in_features) and y + m*ldy (ldy >=
 * out_features), strides in elements; any element alignment is accepted (rows
 * on 16-byte boundaries load wider).  rows == 0 is a no-op.  The workspace is
 * 16-byte aligned and overlaps neither.  bf16 products are exact and summed in fp32 after an
 * offset that is taken out again, so a bf16 row with an infinity gives NaN in
 * every output of that row (finite rows, of whatever size, do not); fp16 and fp32
 * rows follow IEEE arithmetic.  An fp32
 * element enters its products to 2^-23 of itself (one bit less than fp32 has) or
 * 2^-39 of the largest in its 128 inputs, whichever is more: next to inputs 2^16
 * times larger it loses bits even where their weights are 0.
 * Errors: INVALID_ARGUMENT for a NULL handle or pointer, rows < 0, an unknown
 * dtype, a short stride or overlapping buffers; WORKSPACE for a missing or
 * short workspace; HIP when a launch fails. */
bconv_status_t bconv_q4_linear_forward(bconv_q4_linear_t h, void *stream, int32_t rows, int32_t dtype,
                                       const void *x, int64_t ldx, void *y, int64_t ldy, void *workspace,
                                       size_t workspace_bytes);

/* Releases the handle's device memory (no queued call may still use it).  NULL is accepted. */
bconv_status_t bconv_q4_linear_destroy(bconv_q4_linear_t h);

/* ------------------------------------------------------------------------
 * Paged cache of keys and values in 4 bits
 *
 * Per token, key/value head and group of `group` channels (the last may be
 * short) the cache keeps a step s and a midpoint b in fp16, per channel a
 * 4-bit code c; a channel stands for s * (c - 8) + b.  From values x (taken
 * as 0 for NaN, clamped to +-65504), with fp32 operations rounded one by one:
 *   s = fp16((max x - min x) * fp32(1/15)),   b = fp16(min x + 8 s),
 *   c = min(max(rint((x - b) * (1 / s)) + 8, 0), 15)     (c = 8 where s = 0).
 * ------------------------------------------------------------------------ */

typedef struct {
    int32_t num_blocks; /* blocks (pages) of the pool, >= 1; num_blocks * block_size < 2^31 */
    int32_t block_size; /* tokens a block: a power of two, 16 .. 1024 */
    int32_t kv_heads;   /* 1 .. 1024 */
    int32_t head_dim;   /* a multiple of 8, 8 .. 256 */
    int32_t group;      /* channels that share a step: 32, 64 or 128 */
} bconv_kv4_desc_t;

/* Where things are in the pool, in bytes.  Block p, head h has a record of
 * record_bytes at (p * kv_heads + h) * record_bytes, in which token t of the
 * block has
 *   key codes     at t * row_bytes,
 *   value codes   at v_codes_offset + t * row_bytes,
 *   key (s, b)    at k_scales_offset + t * groups * 4, fp16 pairs a group,
 *   value (s, b)  at v_scales_offset + t * groups * 4.
 * dim_padded is head_dim rounded up to 64, 128 or 256; row_bytes =
 * dim_padded / 2.  A row's words, with P = dim_padded:
 *   keys:   word a * P/32 + s (a < 4, s < P/32) holds channels 32 s + 8 a + i,
 *           i < 8: channel i at nibble i/2 + 4 (i % 2), the word then rotated
 *           left by 3 bits;
 *   values: the row is 16 parts of P/16 nibbles, nibble j of part r is channel
 *           16 j + r.
 * A channel of a key row at 32 s + 8 a + i and of a value row at 16 j + r both
 * count from 0; padding channels hold code 8. */
typedef struct {
    size_t pool_bytes, record_bytes;
    int32_t row_bytes, dim_padded, groups, reserved;
    size_t v_codes_offset, k_scales_offset, v_scales_offset;
} bconv_kv4_layout_t;

/* Checks a descriptor and gives the layout (host only, no device). */
bconv_status_t bconv_kv4_layout(const bconv_kv4_desc_t *desc, bconv_kv4_layout_t *layout);

/* Writes `tokens` new rows of keys and values into the pool (device, 16-byte
 * aligned, layout.pool_bytes; clear it once before its first use).  k and v
 * hold elements of `dtype`; channel d of head h of token t is at
 * t*token_stride + h*head_stride + d (strides in elements, each side its own;
 * channels are contiguous; any element alignment).  slots[t] is the token's
 * place, block * block_size + offset; a slot outside the pool (-1 for padding)
 * is not written.  Two tokens must not share a slot.  k_out and v_out, when
 * given, receive the values the cache stands for, in `dtype`, dense
 * [tokens][kv_heads][head_dim], whether or not the token has a slot; they
 * overlap neither k, v nor the pool.
 * tokens == 0 is a no-op. */
bconv_status_t bconv_kv4_append(const bconv_kv4_desc_t *desc, void *stream, void *pool, int32_t tokens,
                                int32_t dtype, const void *k, int64_t k_token_stride, int64_t k_head_stride,
                                const void *v, int64_t v_token_stride, int64_t v_head_stride,
                                const int32_t *slots, void *k_out, void *v_out);

/* Attention over the cache:
 *   out[t][h] = softmax(scale * q[t][h] . K^T + mask) V
 * over the cached keys and values of the token's request and of key/value head
 * h / (heads / kv_heads).  Request r has context_lens[r] cached tokens (its new
 * ones among them), token p of it being row p % block_size of block
 * block_table[r][p / block_size], and queries q_start[r] .. q_start[r+1]-1,
 * which are its last tokens: query j of n sees positions p <= context_lens[r]
 * - n + j, and with a window w > 0 only the last w of those.  Positions whose
 * block id is outside the pool, or past the table's width, are masked.  A
 * query that sees nothing gives 0 (and lse -inf).  Queries of a request past
 * max_q, and past q_tokens, are not computed.
 * Logits, the softmax and all sums are fp32; fp32 queries enter as fp32 rows of a
 * linear layer do (the largest being the query's own).  A probability times its
 * value's step meets the code in 11 bits for bf16 results (fewer where the step is
 * below 2^-19 of the largest that the workgroup's wave has met), 16 bits for fp16
 * results and 23 bits for fp32 results; what it adds to the denominator is fp32. */
typedef struct {
    const void *pool;
    const void *q;               /* [q_tokens][heads][head_dim], strides below (elements) */
    int64_t q_token_stride, q_head_stride;
    void *out;                   /* same shape and type, dense; apart from q, the pool and the workspace */
    float *lse;                  /* [q_tokens][heads] log of the softmax denominators, or NULL */
    const int32_t *block_table;  /* device [requests][table_stride] */
    const int32_t *context_lens; /* device [requests] */
    const int32_t *q_start;      /* device [requests + 1], or NULL: q_tokens / requests queries each */
    int32_t requests, q_tokens;
    int32_t max_q;               /* most queries of one request */
    int32_t heads;               /* a multiple of kv_heads */
    int32_t table_width, table_stride;
    int32_t max_context;         /* most cached tokens of one request (up to 2^30), or 0: the table's width */
    int32_t window;              /* 0: none */
    int32_t dtype;
    float scale;                 /* |scale| below 2^115 */
} bconv_kv4_attention_t;

/* Workspace bytes the call needs (0 is possible); host only. */
bconv_status_t bconv_kv4_attention_workspace_size(const bconv_kv4_desc_t *desc, const bconv_kv4_attention_t *args,
                                                  size_t *bytes);

/* The attention.  max_context and max_q bound device values that the host does
 * not see: keys past max_context are not read, so a bound that is too small
 * loses keys, and workgroups are launched for max_q queries in every request.
 * requests == 0 or q_tokens == 0 is a no-op; without q_start,
 * q_tokens must be a multiple of requests.  Rows of `out` that no request owns
 * are left as they were. */
bconv_status_t bconv_kv4_attention(const bconv_kv4_desc_t *desc, void *stream, const bconv_kv4_attention_t *args,
                                   void *workspace, size_t workspace_bytes);

/* ------------------------------------------------------------------------
 * Block tables and slot maps
 *
 * Request r has context_lens[r] cached tokens and gets new_lens[r] more
 * (negative lengths count as 0).  With have = ceil(context/block_size) and
 * need = min(ceil((context+new)/block_size), table_width), entries have ..
 * need-1 of its table row are filled from free_blocks, requests taking theirs
 * in order from index *free_head on; an entry for which none is left becomes
 * -1.  Outputs:
 *   slots[i], positions[i]  of new token i (requests' tokens one after the
 *                           other): block * block_size + offset, or -1 where
 *                           there is no block; context + index in the request.
 *                           Entries past the last new token get -1 and 0
 *   q_start[requests + 1]   prefix sums of new_lens
 *   context_lens_out        context + new
 *   free_head_out           *free_head + the blocks asked for; more than
 *                           free_count says that some were missing
 * slots, positions, q_start and context_lens_out may each be NULL.  One
 * launch; no result may overlap the table or an input (context_lens_out not
 * context_lens, free_head_out not free_head).  requests at most 8192; with 0, slots, positions,
 * q_start and free_head_out are still written. */
bconv_status_t bconv_block_tables(void *stream, int32_t requests, int32_t block_size, int32_t *block_table,
                                  int32_t table_width, int32_t table_stride, const int32_t *context_lens,
                                  const int32_t *new_lens, const int32_t *free_blocks, int32_t free_count,
                                  const int32_t *free_head, int32_t *free_head_out, int32_t tokens,
                                  int32_t *slots, int32_t *positions, int32_t *q_start,
                                  int32_t *context_lens_out);

#ifdef __cplusplus
}
#endif

#endif /* BCONV_Q4_H */
