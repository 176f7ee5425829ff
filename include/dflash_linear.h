/*
 * dflash_linear.h — C ABI of the matrix product with its epilogue on one GB300
 * GPU: the projections around the attention block and the output head of a
 * verifying model.
 *
 *     y = residual + act(x W^T + bias)
 *
 * for x [rows, k] and W [n, k]: a single token, a draft block's rows or a long
 * prompt's.
 *
 * Conventions: as in dflash_select.h (device pointers owned by the caller,
 * asynchronous on `stream`, no aborts; a non-zero status means nothing was
 * launched and dflash_last_error() has the message). Strides count elements.
 */
#ifndef DFLASH_LINEAR_H
#define DFLASH_LINEAR_H

#include <stdint.h>

#include "dflash_paged.h"
#include "dflash_select.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DFLASH_ACT_NONE = 0,
    DFLASH_ACT_RELU = 1,      /* max(z, 0) */
    DFLASH_ACT_SILU = 2,      /* z / (1 + exp(-z)) */
    DFLASH_ACT_GELU = 3,      /* z (1 + erf(z / sqrt 2)) / 2 */
    DFLASH_ACT_GELU_TANH = 4  /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
} dflash_activation;

/* Shapes fixed for the lifetime of a handle: 1 <= n, k <= 2^30. */
typedef struct {
    int64_t n, k;       /* W [n, k] */
    int64_t w_stride;   /* between W's rows: >= k, a multiple of 8 (any value with n = 1) */
    int32_t dtype;      /* of x, W and bias: DFLASH_BF16 or DFLASH_FP16 */
    int32_t out_dtype;  /* of y and residual: the same, or DFLASH_FP32 */
    int32_t activation; /* dflash_activation */
} dflash_linear_config;

typedef struct dflash_linear_ctx *dflash_linear_handle;

/* A handle for one layer's weights: W [n, k] (16-byte aligned) and bias [n]
 * (or NULL). They are borrowed: they must stay valid and unchanged until
 * dflash_linear_destroy. Waits for `stream`, on which they may just have been
 * written. Holds an error word on the device and no workspace.
 * Errors: INVALID_ARG, UNSUPPORTED (also: not an sm_103 GPU), CUDA. */
dflash_status dflash_linear_init(const dflash_linear_config *cfg, const void *W, const void *bias, void *stream,
                                 dflash_linear_handle *out);

/* y [rows, n] for x [rows, k], 0 <= rows <= 2^30 (0 launches nothing). x is
 * 16-byte aligned and x_stride, the distance of its rows, a multiple of 8 and
 * >= k (any value with one row). y and residual (or NULL) may have any stride
 * >= n and the alignment of their type; rows that start on whole 16 bytes are
 * the fast ones. residual may be y itself (same address and stride, in place);
 * y overlaps nothing else. Products accumulate in fp32 and y is rounded once.
 * The tensor cores' sums truncate: where all products have one sign, an fp32 y
 * is too small by up to 1.1e-6 of itself (bf16) or 3.3e-6 (fp16), with both
 * signs it is nearer; a 16-bit y, before its rounding, by k / 512 times as much
 * for k up to 65536 and by 3e-5 above. Calls give the same bits each time.
 * Calls with one handle may overlap on the GPU. Current device: the handle's.
 * Errors: INVALID_ARG, CUDA. */
dflash_status dflash_linear_run(dflash_linear_handle h, const void *x, int64_t x_stride, int64_t rows,
                                const void *residual, int64_t residual_stride, void *y, int64_t y_stride, void *stream);

/* Waits for `stream` and reports (then clears) the device error word: DFLASH_OK or DFLASH_ERR_TIMEOUT. */
dflash_status dflash_linear_sync_status(dflash_linear_handle h, void *stream);

/* Frees the handle (synchronises its device first). NULL is accepted. */
dflash_status dflash_linear_destroy(dflash_linear_handle h);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_LINEAR_H */
