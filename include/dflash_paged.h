/*
 * dflash_paged.h — C ABI of the attention block around the path selector on
 * one GB300 GPU: the operators that a verifying model (and the drafter's own
 * attention layers) runs on a block's tokens.
 *
 *   dflash_qk_norm_rope  per-head RMS norm and position rotation of queries
 *                        and keys;
 *   dflash_paged_append  the same transform, with the keys and values written
 *                        to a paged cache;
 *   dflash_paged_attend  attention of each sequence's newest tokens (a single
 *                        token, a block of 4 to 16, or a long chunk) over its
 *                        pages.
 *
 * One step of a layer for a batch of B sequences with new[b] tokens each:
 * append (which also transforms the queries), then attend; after the accept
 * check (dflash_verify_prefix) the caller moves lens[b] back to what was
 * kept, and the next append overwrites the rejected rows.
 *
 * Conventions: as in dflash_select.h (device pointers owned by the caller,
 * asynchronous on `stream`, no aborts; a non-zero status means nothing was
 * launched and dflash_last_error() has the message). Strides count elements.
 * Every tensor's last dimension is contiguous; the other strides are
 * multiples of 16 bytes and the base addresses 16-byte aligned.
 */
#ifndef DFLASH_PAGED_H
#define DFLASH_PAGED_H

#include <stdint.h>

#include "dflash_select.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DFLASH_BF16 = 0,
    DFLASH_FP16 = 1,
    DFLASH_E4M3 = 2  /* 8-bit cache: a stored value x stands for x * scale */
} dflash_dtype;

/* Shapes fixed for the lifetime of a handle. Supported: heads a multiple of
 * kv_heads, 1 <= kv_heads <= heads <= 1024; head_dim 64 or 128; page_size a
 * multiple of 16 in [16, 1024]; dtype BF16 or FP16; cache_dtype = dtype or
 * E4M3; 1 <= max_batch <= 65536. */
typedef struct {
    int32_t heads, kv_heads, head_dim, page_size;
    int32_t dtype;        /* of q, k, v and out */
    int32_t cache_dtype;  /* of the cache */
    int32_t max_batch;    /* largest batch any call will pass */
} dflash_paged_config;

/* One layer's cache: keys and values [num_pages, page_size, kv_heads,
 * head_dim] with any strides (so [num_pages, kv_heads, page_size, head_dim]
 * too), the same for both. Only read by dflash_paged_attend. */
typedef struct {
    void *k, *v;
    int64_t num_pages;  /* < 2^31 */
    int64_t page_stride, slot_stride, head_stride;
    float k_scale, v_scale;  /* >= 2^-126, finite; E4M3 caches only (1 is taken otherwise) */
} dflash_paged_cache;

/* The batch of a call. Sequence b has the new tokens cu_tokens[b] ..
 * cu_tokens[b+1]-1 of the call's rows; lens[b] is its length in the cache with
 * them, so new token i has place lens[b] - new[b] + i, and place p is slot
 * p % page_size of page page_table[b][p / page_size]. cu_tokens[0] = 0 and
 * rows from cu_tokens[batch] on are padding: not read, not written. A sequence
 * may have no new tokens. All arrays are int32 on the device and are read by
 * the kernels, so a captured graph can be replayed with other values. */
typedef struct {
    const int32_t *cu_tokens;   /* [batch + 1] */
    const int32_t *lens;        /* [batch] */
    const int32_t *page_table;  /* [batch, table_cols], rows table_stride apart */
    int64_t table_stride;
    int32_t table_cols;
    int32_t batch;       /* 0 <= batch <= max_batch; 0 launches nothing */
    int32_t tokens;      /* rows of q, k, v and out: >= cu_tokens[batch], <= 2^30, tokens * heads < 2^31 */
    int32_t max_tokens;  /* >= every new[b]; picks kernel and tile, the results do not depend on it */
} dflash_paged_batch;

/* Norm and rotation of a head x of head_dim values, in fp32, rounded once:
 *     y = x * w / sqrt(mean(x^2) + eps)     (weights given; else y = x)
 *     (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
 * for the pairs (a, b) = (i, i + rotary_dim/2), or (2i, 2i + 1) with
 * interleaved = 1, i < rotary_dim/2; values from rotary_dim on pass. */
typedef struct {
    const float *table;    /* [positions, rotary_dim] fp32: rotary_dim/2 cosines, then the sines */
    int64_t positions;     /* rows of table, < 2^31; a position outside is clamped and latched */
    int32_t rotary_dim;    /* 0 (no rotation) or a multiple of 16, <= head_dim */
    int32_t interleaved;
    const void *q_weight;  /* [head_dim] of the call's dtype, or NULL */
    const void *k_weight;
    float eps;
} dflash_qk_transform;

typedef struct dflash_paged_ctx *dflash_paged_handle;

/* q [tokens, heads, head_dim] -> q_out, k [tokens, kv_heads, head_dim] ->
 * k_out (either pair may be NULL; in place is allowed, other overlaps are
 * not). dtype BF16 or FP16, head_dim 64, 128 or 256, tokens * heads < 2^31.
 * positions [tokens] int32 (may be NULL with rotary_dim = 0). No handle, no
 * workspace; launched on the current device, which holds all tensors; a position
 * outside the table is clamped silently here.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
dflash_status dflash_qk_norm_rope(const void *q, int64_t q_token_stride, int64_t q_head_stride, void *q_out,
                                  int64_t qo_token_stride, int64_t qo_head_stride, const void *k,
                                  int64_t k_token_stride, int64_t k_head_stride, void *k_out, int64_t ko_token_stride,
                                  int64_t ko_head_stride, int32_t tokens, int32_t heads, int32_t kv_heads,
                                  int32_t head_dim, int32_t dtype, const dflash_qk_transform *transform,
                                  const int32_t *positions, void *stream);

/* Checks the shapes and allocates the workspace that attention over split
 * sequences needs (the only allocation; 40 MB with head_dim 128), cleared on
 * `stream`, which it waits for. One handle serves all layers of a model; its
 * calls must not overlap on the GPU (order them on one stream, any).
 * Errors: INVALID_ARG, UNSUPPORTED (also: not an sm_103 GPU), CUDA. */
dflash_status dflash_paged_init(const dflash_paged_config *cfg, void *stream, dflash_paged_handle *out);

/* Writes k and v [tokens, kv_heads, head_dim] of the batch's new tokens to
 * their places in the cache, k after the transform (NULL: as it is), both
 * divided by their scale (a product with its fp32 reciprocal) and rounded
 * (saturating) for E4M3. With q also q_out = the transformed q [tokens, heads,
 * head_dim] (in place is allowed). A token's position is its place, or
 * positions[token] where given. Keys and values of a token without a valid
 * place or page are not written, and it is latched as DEVICE_CHECK. Errors: INVALID_ARG, CUDA. */
dflash_status dflash_paged_append(dflash_paged_handle h, const dflash_paged_cache *cache,
                                  const dflash_paged_batch *batch, const void *k, int64_t k_token_stride,
                                  int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                                  const dflash_qk_transform *transform, const int32_t *positions, const void *q,
                                  int64_t q_token_stride, int64_t q_head_stride, void *q_out, int64_t qo_token_stride,
                                  int64_t qo_head_stride, void *stream);

/* out [tokens, heads, head_dim] = softmax(scale * q k^T) v of every new token
 * over the keys that it sees: those at places < lens[b] and, with causal = 1,
 * <= its own; with window > 0 only those at places > its own - window. Head j
 * reads key/value head j / (heads / kv_heads). A token that sees no key gets
 * zeros. lse [tokens, heads] fp32 (optional): the natural logarithm of the
 * sum of exp(score), -inf for such a token, NaN (like out) where a score is NaN
 * or +inf. out must not overlap q.
 * Sums, maxima and products accumulate in fp32; the softmax weights are
 * rounded to the cache's 16-bit type (fp16 for E4M3 caches) for the matrix
 * product; in fp16 a weight below 2^-32 of the row's largest counts as zero
 * there. What is stored at places >= lens[b], and on pages that hold no key
 * that some token of the call sees, is never used and may be anything (those
 * pages need no entry in the table). The values (not the keys) at the other
 * places have to be finite for the tokens that do not see them too: their
 * weight there is zero. Keys on an invalid page read as zeros, a length beyond
 * the table is cut to it, and both are latched as DEVICE_CHECK. lens[b] stays
 * below 2^31 - 4096.
 * Errors: INVALID_ARG, CUDA. */
dflash_status dflash_paged_attend(dflash_paged_handle h, const dflash_paged_cache *cache,
                                  const dflash_paged_batch *batch, const void *q, int64_t q_token_stride,
                                  int64_t q_head_stride, void *out, int64_t out_token_stride, int64_t out_head_stride,
                                  float *lse, int32_t causal, int32_t window, float scale, void *stream);

/* Waits for `stream` and reports (then clears) the device error word:
 * DFLASH_OK, DFLASH_ERR_DEVICE_CHECK or DFLASH_ERR_TIMEOUT. */
dflash_status dflash_paged_sync_status(dflash_paged_handle h, void *stream);

/* Frees the handle (synchronises the device first). NULL is accepted. */
dflash_status dflash_paged_destroy(dflash_paged_handle h);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_PAGED_H */
