/*
 * dflash_logits.h — C ABI of what lies between the target model's logits and
 * the accept checks on one GB300 GPU: penalties for repeated tokens, biases and
 * a grammar's mask, and from them the probabilities that
 * dflash_verify_rejection takes, the best tokens that dflash_verify_prefix
 * takes, or the logits themselves.
 *
 * Conventions: as in dflash_select.h (device pointers owned by the caller,
 * asynchronous on `stream`, no aborts; a non-zero status means nothing was
 * launched and dflash_last_error() has the message). Strides count elements.
 */
#ifndef DFLASH_LOGITS_H
#define DFLASH_LOGITS_H

#include <stdint.h>

#include "dflash_paged.h"
#include "dflash_select.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What holds for each sequence of a batch; every array may be NULL (neutral),
 * all are read on the device. Token ids outside [0, vocab) are passed over. */
typedef struct {
    const int32_t *tokens;       /* [batch, token_cols], rows token_stride apart: a sequence's tokens so far, prompt first */
    int64_t token_stride;
    int32_t token_cols;
    const int32_t *lens;         /* [batch] how many; required with tokens; cut to [0, token_cols] */
    const int32_t *prompt_lens;  /* [batch] those of the prompt (NULL: 0) */
    const float *repetition;     /* [batch] rho > 0 */
    const float *presence;       /* [batch] alpha */
    const float *frequency;      /* [batch] beta */
    const float *temperature;    /* [batch] tau >= 0, for the probabilities */
    const int32_t *bias_ids;     /* [batch, bias_count], rows bias_stride apart; an id listed twice: the last one counts */
    const float *bias_values;    /* the same shape and stride */
    int64_t bias_stride;
    int32_t bias_count;
} dflash_logits_rules;

/* Logits [batch, rows, vocab] (dtype BF16, FP16 or DFLASH_FP32; last dimension
 * contiguous): position t of sequence b follows its tokens and draft[b][0 ..
 * t-1] (rows = 1: after the tokens alone). With x a token's logit, seen if it
 * is among those, and c its number of times among those behind the prompt, in
 * fp32, every operation rounded on its own, in this order:
 *     x = x / rho  (x > 0),  x * rho  (otherwise)     if seen
 *     x = x - beta * c,  x = x - alpha                if c > 0
 *     x = x + its bias                                if listed
 *     x = -inf                                        if its mask bit is 0
 * Outputs (NULL = not wanted, but one is):
 *   out    [batch, rows, vocab] of dtype: x, rounded once; may be the logits (same address and strides)
 *   probs  [batch, rows, vocab] fp32, packed: softmax of x / tau over the vocabulary. tau = 0: 1 at the best token.
 *          All 0 where no x is above -inf, all NaN where an x is NaN or +inf (tau > 0).
 *   argmax [batch, rows] int32: the token of the largest x, the lowest id of equals (NaN does not count); -1 where
 *          no x is above -inf
 *   draft  [batch, rows - 1] int32, rows draft_stride apart (NULL with rows = 1, or: no drafts are counted)
 *   mask   int32 words, bit v % 32 of word v / 32 set where token v is allowed: words of position t of sequence b at
 *          mask + b * mask_seq_stride + t * mask_row_stride (a stride of 0 shares them)
 * Outputs overlap nothing else, or the call is refused; rows of out may pass those of the logits where strides are equal
 * (slices of one buffer). 0 <= batch, rows (0 launches nothing), batch * rows < 2^31; vocab >= 1, and what 16
 * CTAs' shared memory holds of it (UNSUPPORTED above): 262,144 tokens with up to 8192 biases, a million and more of
 * 16-bit logits without penalties and biases. Every wait ends within a second.
 * Where a position's logits have not arrived on an SM by then (a fault of the machine), its argmax is -1 (maybe that of the
 * position before it too), its probs are all NaN, and its out is NaN at least where that SM's tokens are; so may be the
 * sequence's positions behind it. No handle, no workspace; launched on
 * the current device.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
dflash_status dflash_logits_adjust(const void *logits, int64_t seq_stride, int64_t row_stride, int32_t batch, int32_t rows,
                                   int64_t vocab, int32_t dtype, const dflash_logits_rules *rules, const int32_t *draft,
                                   int64_t draft_stride, const int32_t *mask, int64_t mask_seq_stride,
                                   int64_t mask_row_stride, void *out, int64_t out_seq_stride, int64_t out_row_stride,
                                   float *probs, int32_t *argmax, void *stream);

/* Self-test of that: dflash_logits_adjust on packed logits, but copies of the logits do not come for one CTA, `rank` of the
 * first cluster, from the cluster's position `at` on (a cluster takes positions of the first sequence; without such a CTA or
 * position, or for rows that threads bring, nothing is lost). Takes some seconds. Errors: as above. */
dflash_status dflash_selftest_logits_lost(const void *logits, int32_t batch, int32_t rows, int64_t vocab, int32_t dtype,
                                          const dflash_logits_rules *rules, void *out, float *probs, int32_t *argmax,
                                          int32_t rank, int32_t at, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_LOGITS_H */
