/*
 * eqlinear_rmsnorm.h -- C ABI of the equivariant RMS norm with the residual's addition, forward and
 * backward, in the same library: the norm of pre-norm blocks that do without a mean and a bias.
 *
 * Conventions, sizes, types and status codes are eqlinear.h's: device pointers, 16-byte aligned unless
 * said otherwise, dense row-major arrays of `dtype`, everything asynchronous on `stream`, arguments
 * checked before anything is launched.  Rows have R = C'*T features, flat index c*T + t.  Sums and
 * what is computed in between are fp32; every conversion to `dtype` rounds to nearest even.  Results
 * do not depend on timing: sums are added in a fixed order.
 */
#ifndef EQLINEAR_RMSNORM_H
#define EQLINEAR_RMSNORM_H

#include "eqlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * RMS norm of each row with the residual's addition, one weight per channel, shared by its T group
 * elements (T = 1 is the ordinary one):
 *     s = x + residual, rounded to `dtype`;  rstd = 1 / sqrt(mean(s^2) + eps),
 *     y[n][c*T+t] = gamma[c] s rstd
 * The norm is of the rounded sum: what `sum` receives is what the backward pass reads.
 * x, residual: [N][Cp*T] read; residual may be NULL (s = x).  gamma: [Cp] of `dtype`, or NULL (1),
 *   aligned to the element.
 * sum: [N][Cp*T] written, or NULL; may be x or residual.  y: [N][Cp*T] written; may be x or residual,
 *   but not sum (EQL_EINVAL).
 * rstd: [N] floats, or NULL (4-byte aligned); the backward pass needs it.
 * eps: >= 0 and finite, else EQL_EINVAL.  A row whose s holds an infinity or a NaN, or whose squares
 *   overflow fp32, or whose mean square + eps is 0 or below fp32's normal range, gives NaN throughout
 *   (s itself is as added).
 * Rows over 16384 features take N <= 2^22 - 1 (EQL_EINVAL otherwise).
 */
int eqlinear_rmsnorm_fwd(const void* x, const void* residual, const void* gamma, void* sum, void* y, float* rstd,
                         int64_t N, int64_t Cp, int T, float eps, int dtype, void* stream);

/* Scratch bytes of its backward (0 when N == 0 or the arguments are invalid): fp32 column sums per block
 * of rows, and for rows over 8192 features two floats a row. */
size_t eqlinear_rmsnorm_bwd_workspace_bytes(int64_t N, int64_t Cp, int T, int dtype);

/*
 * Backward of eqlinear_rmsnorm_fwd.  With g = dy gamma[c] and h = s rstd:
 *     dx        = rstd (g - h mean(g h)) + dres      (the gradient of x, and of the residual)
 *     dgamma[c] = sum over n and t of dy h
 * dy, sum (the forward's s: sum, or x without a residual), dres: [N][Cp*T] read; dres: the gradient
 * that reaches s by the residual stream, or NULL.  rstd: the forward's.  dx: [N][Cp*T] written, may be
 * dy or dres.  dgamma: [Cp] of `dtype`, or NULL (zeros when N == 0), aligned to the element.
 * workspace: eqlinear_rmsnorm_bwd_workspace_bytes bytes (rows up to 8192 features need none when
 * dgamma is NULL).  The column sums add fp32 products in an order
 * fixed by N, Cp and T.  Rows over 8192 features take N <= 2^22 - 1.
 */
int eqlinear_rmsnorm_bwd(const void* dy, const void* sum, const float* rstd, const void* gamma, const void* dres,
                         void* dx, void* dgamma, void* workspace, size_t ws_bytes, int64_t N, int64_t Cp, int T,
                         int dtype, void* stream);

/* Version of this header (major * 100 + minor). */
int eqlinear_rmsnorm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* EQLINEAR_RMSNORM_H */
