/*
 * ssm_group_norm.h -- C ABI of libssm: the norm of groups of a token's channels
 * (the heads of an attention's or a scan's output) with an activation or a gate,
 * forward and backward, on AMD Instinct MI355X (gfx950).
 *
 * For each token and each of `groups` groups of dim / groups consecutive channels:
 *
 *   mean     = average of the group's x
 *   rstd     = 1 / sqrt(average of (x - mean)^2 + eps)
 *   n        = (x - mean) * rstd * weight[d] + bias[d]
 *   y        = n * act(z)        with a gate z
 *            = act(n)            without
 *
 * act is the identity (SSM_ACT_NONE), silu (SSM_ACT_SILU) or the logistic function
 * (SSM_ACT_SIGMOID).  The backward, with xhat = (x - mean) rstd:
 *
 *   dn       = dy * act(z)       or dy * act'(n)
 *   dz       = dy * n * act'(z)
 *   dx       = rstd * (dn w - mean(dn w) - xhat * mean(dn w xhat)),  means over the group
 *   dweight  = sum over tokens of dn * xhat
 *   dbias    = sum over tokens of dn
 *
 * Conventions as in ssm.h (device pointers, stream, validation before any HIP
 * call, aliasing judged on byte ranges, deterministic results), and:
 *  - x, z, y, dy, dx, dz: (tokens, dim), dtype, channels last; x and z may have
 *    rows apart (x_stride, z_stride, elements from one token to the next: a block of
 *    a wider projection's output), the others are contiguous.  mean, rstd:
 *    (tokens, groups) float32; weight, bias, dweight, dbias: (dim) float32.
 *    Pointers need their element's alignment only.
 *  - Every sum is held in float32 or wider, the variance taken about the mean;
 *    outputs are rounded once.  A group of equal values has exactly that mean and
 *    variance 0: n is the bias (NaN where eps is 0 too).  Deviations may be of any
 *    size, past float32's range too (a group partly at the type's lowest value):
 *    rstd may then be subnormal, with its fewer bits, and the backward has these.
 *  - A NaN or Inf in one group makes that group NaN where the formula does and
 *    leaves the others alone.
 */
#ifndef SSM_GROUP_NORM_H
#define SSM_GROUP_NORM_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { SSM_ACT_NONE = 0, SSM_ACT_SILU = 1, SSM_ACT_SIGMOID = 2 } ssm_act_t;

/* Most channels of a group. */
#define SSM_GROUP_NORM_MAX_WIDTH 8192

/*
 * ssm_group_norm_fwd
 *   x            in   required
 *   x_stride     >= dim
 *   weight, bias in   (dim) float32, NULL -> 1 and 0
 *   z            in   NULL -> no gate
 *   z_stride     >= dim with z
 *   act          one of ssm_act_t (SSM_ERR_FLAGS otherwise)
 *   eps          >= 0 and finite (SSM_ERR_SHAPE otherwise)
 *   y            out  required; must overlap no other buffer of the call
 *   mean, rstd   out  NULL -> not written
 *   tokens >= 0, dim >= 1, groups >= 1 and dividing dim, dim / groups at most 8192,
 *   tokens * groups at most 2^31 - 4097, strides at most 2^31 - 1 (SSM_ERR_SHAPE
 *   otherwise).
 */
int ssm_group_norm_fwd(const void* x, int64_t x_stride, const float* weight, const float* bias,
                       const void* z, int64_t z_stride, int act, float eps, void* y, float* mean,
                       float* rstd, int64_t tokens, int dim, int groups, int dtype, void* stream);

/*
 * ssm_group_norm_bwd
 *   x .. act     in   as for ssm_group_norm_fwd (the same values)
 *   mean, rstd   in   (tokens, groups) float32, from the forward pass; required
 *   dy           in   required
 *   dx           out  required
 *   dz           out  required with z
 *   dweight      out  (dim) float32                             NULL -> not written
 *   dbias        out  (dim) float32                             NULL -> not written
 *   workspace    at least ssm_group_norm_bwd_workspace_bytes(...) bytes,
 *                256-byte aligned, owned by the caller (NULL where the query
 *                returns 0); calls sharing one workspace must not overlap
 * tokens == 0 writes zeros to dweight and dbias.
 */
int ssm_group_norm_bwd(const void* x, int64_t x_stride, const float* weight, const float* bias,
                       const void* z, int64_t z_stride, int act, const float* mean,
                       const float* rstd, const void* dy, void* dx, void* dz, float* dweight,
                       float* dbias, int64_t tokens, int dim, int groups, int dtype, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Bytes of device workspace of ssm_group_norm_bwd (sums of dweight and dbias over
 * part of the tokens).  Pure host function; 0 for an empty problem and for
 * arguments that it would refuse. */
size_t ssm_group_norm_bwd_workspace_bytes(int64_t tokens, int dim, int groups, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* SSM_GROUP_NORM_H */
