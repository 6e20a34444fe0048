/*
 * ssm_norm.h -- C ABI of libssm: layer norm over the channels, forward and
 * backward, on AMD Instinct MI355X (gfx950).
 *
 *   s        = x                          (residual NULL)
 *            = x + residual, rounded to the storage type: the residual stream as the
 *              next block reads it; the norm is taken of the rounded value
 *   mean     = (1/dim) sum_d s
 *   rstd     = 1 / sqrt((1/dim) sum_d (s - mean)^2 + eps)
 *   y        = (s - mean) * rstd * weight[d] + bias[d]
 *
 * and, with xhat = (s - mean) rstd and dn = dy * weight,
 *
 *   dx       = rstd * (dn - mean_d(dn) - xhat * mean_d(dn * xhat)) [+ dsum]
 *   dweight  = sum over batch and steps of dy * xhat
 *   dbias    = sum over batch and steps of dy
 *
 * Conventions as in ssm.h (device pointers, stream, validation before any HIP
 * call, aliasing judged on byte ranges, deterministic results), and:
 *  - x, residual, sum_out, y, dy, dsum, dx: (batch, dim, seqlen), dtype, L
 *    fastest, as the scans' tensors; tokens whose channels lie together,
 *    (tokens, dim), are batch = tokens, seqlen = 1.  mean, rstd:
 *    (batch, seqlen) float32; weight, bias, dweight, dbias: (dim) float32.
 *    Contiguous; pointers need their element's alignment only.
 *  - Every sum is held in float32 or wider, the variance taken about the mean;
 *    y and dx are rounded once.  A token of equal values has exactly that mean
 *    and variance 0: y is the bias (NaN where eps is 0 too).  Where the squares
 *    of a token's deviations pass float32's range, rstd is 0 and y the bias
 *    (or NaN, where a deviation passes it itself).
 *  - A NaN or Inf in one token makes that token's y (and dx) NaN where the
 *    formula does and leaves the other tokens alone.
 */
#ifndef SSM_NORM_H
#define SSM_NORM_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ssm_layer_norm_fwd
 *   x            in   required
 *   residual     in   NULL -> none; may be x
 *   weight       in   (dim) float32, required
 *   bias         in   (dim) float32, NULL -> 0
 *   eps          >= 0 and finite (SSM_ERR_SHAPE otherwise)
 *   y            out  required; must overlap no other buffer of the call
 *   sum_out      out  required with residual, refused (SSM_ERR_NULL) without; must
 *                     overlap no other buffer of the call
 *   mean, rstd   out  NULL -> not written
 *   batch, seqlen >= 0, seqlen at most 2^31 - 4097; dim >= 1; batch * seqlen at
 *   most 2^31 - 4097 where seqlen < 8 or a row has 2^31 bytes, batch * seqlen / 8
 *   elsewhere (SSM_ERR_SHAPE otherwise).
 */
int ssm_layer_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias,
                       float eps, void* y, void* sum_out, float* mean, float* rstd, int batch,
                       int dim, int64_t seqlen, int dtype, void* stream);

/*
 * ssm_layer_norm_bwd
 *   s            in   what was normalised (x, or sum_out)       required
 *   weight       in   (dim) float32                             required
 *   mean, rstd   in   (batch, seqlen) float32, from the forward pass; required
 *   dy           in   required
 *   dsum         in   the gradient arriving at sum_out by the other way; NULL -> none
 *   dx           out  the gradient of x, and of residual        required
 *   dweight      out  (dim) float32                             required
 *   dbias        out  (dim) float32                             NULL -> not written
 *   workspace    at least ssm_layer_norm_bwd_workspace_bytes(...) bytes,
 *                256-byte aligned, owned by the caller (NULL where the query
 *                returns 0); calls sharing one workspace must not overlap
 * batch == 0 or seqlen == 0 writes zeros to dweight and dbias.
 */
int ssm_layer_norm_bwd(const void* s, const float* weight, const float* mean, const float* rstd,
                       const void* dy, const void* dsum, void* dx, float* dweight, float* dbias,
                       int batch, int dim, int64_t seqlen, int dtype, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Bytes of device workspace of ssm_layer_norm_bwd (sums of dweight and dbias
 * over part of the tokens).  Pure host function; 0 for an empty problem and for
 * arguments that it would refuse. */
size_t ssm_layer_norm_bwd_workspace_bytes(int batch, int dim, int64_t seqlen, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* SSM_NORM_H */
