/*
 * eqlinear_block.h -- C ABI of the operators around the EQ-Linear layer in a transformer
 * block, in the same library: an equivariant layer norm, forward and backward, and 8-bit
 * activation checkpoints with the backward passes that read them.
 *
 * The networks the layer is built into ("Nivel de Rede" in "Resumo Tecnico: Flash EQ-Linear":
 * Flash EQ-ViT and Flash EQ-Swin) use it in pre-norm MLP blocks,
 *     y = x + W2 gelu(W1 norm(x) + b1) + b2,
 * and training one keeps the normalised rows and GELU's input from the forward to the backward
 * pass.  With these entry points both are kept in 8 bits and nothing else is:
 *   forward   eqlinear_layernorm_fwd (ckpt: the normalised rows), eqlinear_fwd_fused with
 *             pre_out, eqlinear_ckpt8_pack (pre), eqlinear_fwd_fused with the residual
 *   backward  second layer: eqlinear_bwd_x_train, and its weight gradient from gelu(pre);
 *             eqlinear_fused_epilogue_bwd_ckpt8; first layer: eqlinear_bwd_x_train, and its
 *             weight gradient from gamma h + beta; eqlinear_layernorm_bwd_ckpt8.
 *
 * Conventions, sizes, types and status codes are eqlinear.h's: device pointers, 16-byte aligned
 * unless said otherwise, dense row-major arrays of `dtype`, everything asynchronous on
 * `stream`, arguments checked before anything is launched.  Rows have R = C'*T features, flat
 * index c*T + t.  Sums, statistics and what is computed in between are fp32; every conversion
 * to `dtype` rounds to nearest even.  Results do not depend on timing: sums are added in a
 * fixed order.
 */
#ifndef EQLINEAR_BLOCK_H
#define EQLINEAR_BLOCK_H

#include "eqlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * 8-bit checkpoint of an [N][R] matrix.  32 consecutive features of a row (the row's last block
 * may be shorter) share one power-of-two step 2^e:
 *     e     the smallest integer >= -126 with max|v| 2^-e < 127.5 over the block, but at most 121
 *           (9 where a fp16 matrix is packed): a block of finite values stays finite in its type
 *     code  v 2^-e rounded to nearest even, held to [-127, 127];  value = code 2^e
 * The error is at most half a step, or where the limit on e takes effect (max|v| of 127.5 2^121, in
 * fp16 65280, or more) less than one; at most max|v| / 127 either way.  Codes do not depend on how
 * they are computed.  A block with an infinity or a NaN reads back as NaN throughout.
 * Layout, with P = 32 ceil(R / 32): N rows of P signed bytes (codes; zero past R), then N rows
 * of P / 32 bytes e + 127 (255: the block is NaN, its codes are unspecified).  The size does not
 * depend on the element type, nor does the content for equal values but for fp16's limit on e.
 */
size_t eqlinear_ckpt8_bytes(int64_t N, int64_t Cp, int T);

/* x: [N][Cp*T] read; ckpt: eqlinear_ckpt8_bytes(N, Cp, T) bytes written.  N P <= 2^35 - 2^11 here and
 * in eqlinear_ckpt8_unpack (EQL_EINVAL otherwise). */
int eqlinear_ckpt8_pack(const void* x, void* ckpt, int64_t N, int64_t Cp, int T, int dtype, void* stream);

/* ckpt read; x: [N][Cp*T] written (the values, rounded to `dtype`: exact in fp32, and in fp16
 * where a fp16 matrix was packed whose largest magnitude in the block is at least 2^-18 or so; a
 * fp32 matrix's values may be beyond fp16's range). */
int eqlinear_ckpt8_unpack(const void* ckpt, void* x, int64_t N, int64_t Cp, int T, int dtype, void* stream);

/*
 * Layer norm of each row, with one weight and bias per channel, shared by its T group elements
 * (the statistics run over the whole row, so the norm commutes with the group action; T = 1 is
 * the ordinary layer norm):
 *     h = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),  y[n][c*T+t] = gamma[c] h + beta[c]
 * var is the mean square of the centred row.
 * x: [N][Cp*T] read; y: [N][Cp*T] written, may be x.  gamma, beta: [Cp] of `dtype`, or NULL
 *   (1, 0); aligned to the element.
 * ckpt: eqlinear_ckpt8_bytes(N, Cp, T) bytes, or NULL: receives h as an 8-bit checkpoint
 *   (quantised from fp32).
 * mean, rstd: [N] floats, or NULL (4-byte aligned); the backward pass needs rstd, and mean
 *   unless it reads the checkpoint.
 * eps: >= 0 and finite, else EQL_EINVAL.  A row that holds an infinity or a NaN, or whose
 *   sum or squares overflow fp32, or whose var + eps is 0 or below fp32's normal range, gives NaN
 *   throughout.
 * Rows over 16384 features take N <= 2^22 - 1 (EQL_EINVAL otherwise).
 */
int eqlinear_layernorm_fwd(const void* x, const void* gamma, const void* beta, void* y, void* ckpt, float* mean,
                           float* rstd, int64_t N, int64_t Cp, int T, float eps, int dtype, void* stream);

/* Scratch bytes of the norm's backward (0 when N == 0 or the arguments are invalid): fp32
 * column sums per block of rows, and for rows over 8192 features two floats a row. */
size_t eqlinear_layernorm_bwd_workspace_bytes(int64_t N, int64_t Cp, int T, int dtype);

/*
 * Backward of eqlinear_layernorm_fwd.  With g = dy gamma[c] and h as above:
 *     dx        = rstd (g - mean(g) - h mean(g h)) + dres
 *     dgamma[c] = sum over n and t of dy h,   dbeta[c] = sum over n and t of dy
 * eqlinear_layernorm_bwd takes h from x and the forward's mean and rstd;
 * eqlinear_layernorm_bwd_ckpt8 from the forward's checkpoint (h is then the checkpoint's value
 * everywhere above).
 * dy, x, dres: [N][Cp*T] read; dres: the residual branch's gradient, added to dx, or NULL.
 * dx: [N][Cp*T] written, may be dy or dres.  dgamma, dbeta: [Cp] of `dtype`, or NULL (zeros when
 * N == 0), aligned to the element.  workspace: eqlinear_layernorm_bwd_workspace_bytes bytes
 * (rows up to 8192 features need none when dgamma and dbeta are NULL).  The column sums add
 * fp32 products in an order fixed by N, Cp and T.  Rows over 8192 features take N <= 2^22 - 1.
 */
int eqlinear_layernorm_bwd(const void* dy, const void* x, const float* mean, const float* rstd, const void* gamma,
                           const void* dres, void* dx, void* dgamma, void* dbeta, void* workspace, size_t ws_bytes,
                           int64_t N, int64_t Cp, int T, int dtype, void* stream);
int eqlinear_layernorm_bwd_ckpt8(const void* dy, const void* ckpt, const float* rstd, const void* gamma,
                                 const void* dres, void* dx, void* dgamma, void* dbeta, void* workspace,
                                 size_t ws_bytes, int64_t N, int64_t Cp, int T, int dtype, void* stream);

/*
 * eqlinear_fused_epilogue_bwd with EQL_ACT_GELU and the activation's input read from a
 * checkpoint of [N][Dp*T]:  dpre = dy GELU'(value),  dbias[d] = sum over n and g of dpre.
 * dpre may be dy; dbias may be NULL; workspace as eqlinear_fused_epilogue_bwd's
 * (eqlinear_fused_epilogue_bwd_workspace_bytes bytes when dbias is given).
 */
int eqlinear_fused_epilogue_bwd_ckpt8(const void* dy, const void* pre_ckpt, void* dpre, void* dbias, void* workspace,
                                      size_t ws_bytes, int64_t N, int64_t Dp, int T, int dtype, void* stream);

/*
 * Weight gradient with the layer's input read from a checkpoint of [N][Cp*T]:
 *     x[n][c*T+t] = act(gamma[c] value + beta[c])
 * gamma, beta: [Cp] of `dtype`, or NULL (1, 0), aligned to the element; act: EQL_ACT_NONE or
 * EQL_ACT_GELU (any other value is EQL_EINVAL).  x is formed in fp32 and transformed; only its
 * spectrum is rounded to `dtype` (as dy's; fp16: 4e-4 of the gradient's norm off, where its own last
 * rounding is 2e-4).  The rest as eqlinear_bwd_w, with the same two paths and the
 * same workspace (eqlinear_bwd_w_workspace_bytes) or a larger one: with more, a layer of few rows or
 * channels is split into more row ranges, each with partial sums of its own (232 rows, 22 x 804
 * channels, T = 4, fp32: 54 us with that many bytes, 20 with 3 MB more).  32 MiB more has been
 * enough for any size tried.  The order of the sum depends on the sizes and on ws_bytes, on nothing
 * else.
 */
int eqlinear_bwd_w_ckpt8(const void* ckpt, const void* gamma, const void* beta, int act, const void* dy, void* dw,
                         void* workspace, size_t ws_bytes, int64_t N, int64_t Cp, int64_t Dp, int T, int dtype,
                         void* stream);

/*
 * Only that input's half spectrum, into its place in the weight-gradient workspace: what
 * eqlinear_fwd_train leaves there.  A training step that kept a checkpoint instead of the
 * workspace calls this before or after eqlinear_bwd_x_train (on the same workspace), then
 * eqlinear_bwd_w_train; the contract is eqlinear_bwd_w_train's.
 */
int eqlinear_ckpt8_spectrum(const void* ckpt, const void* gamma, const void* beta, int act, void* workspace,
                            size_t ws_bytes, int64_t N, int64_t Cp, int64_t Dp, int T, int dtype, void* stream);

/* Version of this header (major * 100 + minor). */
int eqlinear_block_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* EQLINEAR_BLOCK_H */
