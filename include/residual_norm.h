/*
 * residual_norm.h -- C ABI of the norm between two blocks in libwkv7, on
 * MI355X (gfx950): the residual sum after a block, with its scale, and the
 * root-mean-square norm before the next one, in one pass.
 *
 *     x_out = x + scale * y          (scale NULL: x + y;  y NULL: x_out = x)
 *     h     = x_out / sqrt(mean(x_out^2) + eps) * w
 *
 * x, y, x_out, h and their gradients are [rows][D] of `dtype`; w, scale, dw
 * and dscale are [D] fp32.  h is formed from the sum before it is rounded to
 * x_out.  The backward takes x_out as it was stored and returns
 *     dx     = dx_out + the gradient of h with respect to x_out
 *     dy     = scale * dx
 *     dw     = sum over rows of dh * x_out / sqrt(..)
 *     dscale = sum over rows of dx * y
 * (without a scale, dy is dx).  The sums over rows run in a fixed order:
 * results are the same bit for bit from run to run.
 *
 * Any D from 1 to 16384 and any number of rows that memory holds (up to 2^38);
 * pointers 16-byte aligned (rows need not be).  Ownership, execution and errors as for wkv7.h.
 */
#ifndef RESIDUAL_NORM_H
#define RESIDUAL_NORM_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t rows;   /* >= 0 */
    int64_t D;      /* 1 to 16384 */
    int32_t dtype;  /* wkv7_dtype */
    int32_t flags;  /* 0 */
    float eps;      /* > 0, finite */
} residual_norm_shape;

size_t residual_norm_workspace_bytes(const residual_norm_shape *shape);

/* x, w, h required; y, scale, x_out may be NULL (scale needs y; x_out may be
 * x itself: the residual stream is updated in place). */
int residual_norm_forward(const residual_norm_shape *shape, const void *x, const void *y,
                          const float *scale, const float *w, void *x_out, void *h,
                          hipStream_t stream);

/* dh, x_out, w, dx, dw required; dx_out NULL = zeros; scale, y, dy and
 * dscale come together or are all NULL.  dx may be dx_out itself.
 * workspace: 256-byte aligned. */
int residual_norm_backward(const residual_norm_shape *shape, const void *dh, const void *dx_out,
                           const void *x_out, const void *y, const float *scale, const float *w,
                           void *dx, void *dy, float *dw, float *dscale, void *workspace,
                           size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RESIDUAL_NORM_H */
