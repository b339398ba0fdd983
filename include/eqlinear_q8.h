/*
 * eqlinear_q8.h -- C ABI of the EQ-Linear layer in 8-bit integers, in the same library: the inference
 * form of a layer, and of the norm in front of it.
 *
 * The layer is a channel product for each frequency of the group axis (eqlinear.h); here the products
 * run on 8-bit integer codes of the half spectrum with 32-bit integer sums, a scale for each row and
 * frequency of the activations, and one for each output channel and frequency of the weight:
 *     once      eqlinear_q8_pack_weight
 *     a call    eqlinear_q8_quantize, or in a pre-norm block eqlinear_q8_rmsnorm (residual addition,
 *               RMS norm and 8-bit output in one pass); then eqlinear_q8_fwd
 * With T = 1 it is the ordinary linear layer with a scale for each token and each output channel.
 *
 * 8-bit form of a vector of channels (a row, or an output channel's weights), from its planes
 *     k = 0: sum_t v_t;   k = T/2 (even T): sum_t (-1)^t v_t;   else Re, Im of sum_t v_t exp(-2 pi i t k / T)
 * Each frequency k takes m = max over the channels of |Re| and |Im|, at least 2^-100;
 *     code = plane * (127 * (1 / m)), each operation rounded to fp32, then to an integer (ties to even):
 *            in [-127, 127];   scale = m / 127.
 * A value of a plane is off by half a scale at most (1 / 254 of the largest of its frequency), and the
 * layer's output by what those errors add up to; the sums are exact.  A cyclic shift of the group axis
 * leaves T = 1, 2 and 4 exactly equivariant (it permutes and negates the codes); other T rotate a
 * complex pair, which the rounding follows to its half step.  An infinity or a NaN in a row makes the
 * row's outputs NaN (also where a plane of finite values overflows fp32); in the weight, that output
 * channel's.
 *
 * Conventions, types and status codes are eqlinear.h's: device pointers, 16-byte aligned unless said
 * otherwise, dense row-major arrays of `dtype`, everything asynchronous on `stream`, arguments checked
 * before anything is launched.  Sizes too, with Cp <= 65536 (EQL_EUNSUPPORTED above: the integer sums
 * would leave 32 bits).  Results do not depend on timing; a row's outputs depend on that row alone, not on N
 * or on the other rows.  These are inference forms: nothing here has a backward pass.
 */
#ifndef EQLINEAR_Q8_H
#define EQLINEAR_Q8_H

#include "eqlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Bytes of N 8-bit rows of Cp*T features (0 for invalid arguments): with P = 16 ceil(Cp / 16) and F =
 * floor(T / 2) + 1, N rows of T planes of P codes (zero past Cp; planes in the order k = 0, T/2 (even T),
 * then Re and Im of k = 1, 2, ...), then N rows of F float scales (k = 0, T/2, 1, 2, ...).
 */
size_t eqlinear_q8_rows_bytes(int64_t N, int64_t Cp, int T);

/* x: [N][Cp*T] read; rows8: eqlinear_q8_rows_bytes(N, Cp, T) bytes written.  Some rows over 6144 features (those
 * that a workgroup's registers do not hold) take N <= 2^24 - 1 (EQL_EINVAL otherwise), here and below. */
int eqlinear_q8_quantize(const void* x, void* rows8, int64_t N, int64_t Cp, int T, int dtype, void* stream);

/*
 * eqlinear_rmsnorm_fwd (eqlinear_rmsnorm.h) with its output in 8 bits: rows8 receives gamma[c] s rstd,
 * formed in fp32 (codes from the planes of s times gamma, rstd in the scales), for s = x + residual
 * rounded to `dtype`.  residual, gamma and sum may be NULL; sum may be x or residual.  eps as there.
 */
int eqlinear_q8_rmsnorm(const void* x, const void* residual, const void* gamma, void* sum, void* rows8, int64_t N,
                        int64_t Cp, int T, float eps, int dtype, void* stream);

/* Bytes of a packed weight (0 for invalid arguments): about Dp*Cp*T, padded to 32 output and 64 input
 * channels.  Its layout is the kernels' own. */
size_t eqlinear_q8_weight_bytes(int64_t Dp, int64_t Cp, int T);

/* w: [Dp][Cp][T] read; w8: eqlinear_q8_weight_bytes(Dp, Cp, T) bytes written, for any N. */
int eqlinear_q8_pack_weight(const void* w, void* w8, int64_t Dp, int64_t Cp, int T, int dtype, void* stream);

/*
 * y[n][d*T+g] = act(layer + bias[d]) + residual, the epilogue in fp32 and rounded once.  GELU
 * is v Phi(v) within 2.5e-7, and below zero within 6e-5 of it down to v = -5.6, past which it lies between -6e-8 and 0.
 * rows8, w8: as written by the calls above for these sizes.  bias: [Dp] of `dtype`, or NULL, aligned to
 * the element; act: EQL_ACT_NONE or EQL_ACT_GELU (any other value is EQL_EINVAL); residual: [N][Dp*T], or NULL,
 * may be y.  y: [N][Dp*T] written.  N and Dp that take 2^24 workgroups or more (each at least 32 rows by 32
 * channels) are EQL_EINVAL.
 */
int eqlinear_q8_fwd(const void* rows8, const void* w8, const void* bias, const void* residual, void* y, int64_t N,
                    int64_t Cp, int64_t Dp, int T, int dtype, int act, void* stream);

/* Version of this header (major * 100 + minor). */
int eqlinear_q8_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* EQLINEAR_Q8_H */
