/*
 * ssm_gated.h -- C ABI of libssm: a gated linear recurrence with one state
 * per channel, its backward pass and its one-token step, on AMD Instinct
 * MI355X (gfx950).
 *
 * The operation (one independent channel per (b, d); all tensors row-major):
 *
 *   g_t = sigmoid(r[b,d,t] + r_bias[d])            (the default)
 *       = softplus(r[b,d,t] + r_bias[d])           (flags & SSM_GATE_SOFTPLUS)
 *   a_t = exp(A[d] * g_t)
 *   w_t = 1 - a_t                                  (the default: h is a convex sum of its inputs)
 *       = sqrt(1 - a_t^2)                          (flags & SSM_GATE_UNIT: unit-variance inputs give a unit-variance h)
 *   u_t = x[b,d,t] * sigmoid(i[b,d,t] + i_bias[d])  (x alone where i is NULL)
 *   h_t = a_t * h_{t-1} + w_t * u_t                (h_{t-1} taken as 0 where starts[b,t] is not 0)
 *   y[b,d,t] = h_t * silu(z[b,d,t])                (h_t alone where z is NULL)
 *
 * With SSM_GATE_SOFTPLUS and A = -1 the decay is sigmoid(-r) and the rule is
 * h = (1 - G) h + G u with G = sigmoid(r): the gated recurrence that the
 * selective scan of one state reduces to ("Paper: Mamba" course module,
 * konke.bhala.ai/m/F12, Theorem 1).  In general it is the selective scan with
 * one state per channel, the step Delta = g, the zero-order-hold decay, and
 * the input weight normalised by its steady-state gain.
 *
 * Conventions as in ssm.h (device pointers, stream, validation before any HIP
 * call, aliasing judged on byte ranges, deterministic results), and:
 *  - dtype (SSM_F32 or SSM_BF16) selects the storage of x, r, i, z, y and
 *    their gradients.  A, the biases and the states are float32; h and every
 *    sum are held in float32 or wider and rounded once.
 *  - x, r, i, z, y, dy, dx, dr, di, dz: (batch, dim, seqlen), L fastest; A,
 *    r_bias, i_bias and their gradients: (dim); h0, last_state, dh0,
 *    dlast_state, state: (batch, dim).  Contiguous.
 *  - starts: (batch, seqlen) bytes, not 0 at the first step of each sequence
 *    packed into a row (a row may begin in the middle of one).  No state, no
 *    gradient and no NaN or Inf crosses a start.  NULL -> none.
 *  - Pointers need their element's alignment only; rows of any length and
 *    alignment take the same vector accesses.
 *  - A padded batch: a step with r = -inf or the type's lowest value (and
 *    finite x and z, and no NaN in i) is the identity, a_t = 1 and w_t = 0,
 *    under either gate, so last_state and the gradients are those of the steps
 *    before it.
 *  - A is not checked for sign; A > 0 grows (and w_t is then negative, or NaN
 *    with SSM_GATE_UNIT), and a state that leaves float32's range is infinite
 *    from there on (a decay that does so in one step is infinite, and NaN times
 *    a state of 0).  Channels whose decays might multiply past 2^100 over 512
 *    steps (A > 0.135 with a sigmoid) are scanned a step at a time, up to 45
 *    times slower.  A decay that underflows is held at the smallest normal
 *    float, so an infinite state stays infinite until the next start.
 *  - Where w_t = 0 under SSM_GATE_UNIT (A g = 0), the square root's infinite
 *    slope is taken as 0 in the backward pass.
 */
#ifndef SSM_GATED_H
#define SSM_GATED_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of the `flags` argument (others: SSM_ERR_FLAGS). */
typedef enum {
  SSM_GATE_SOFTPLUS = 1, /* g = softplus(r + r_bias), else sigmoid */
  SSM_GATE_UNIT = 2      /* w = sqrt(1 - a^2), else 1 - a          */
} ssm_gate_flag_t;

/* Steps between two kept states of the forward pass (ckpt). */
#define SSM_GATED_CKPT_STEPS 512

/* Bytes of the kept states of a scan: h entering every
 * SSM_GATED_CKPT_STEPS-th step, (batch, ceil(seqlen / 512), dim) float32 (the
 * first is h0, or zero).  Pure host function; 0 for an empty problem and for
 * sizes the scan would refuse. */
size_t ssm_gated_scan_ckpt_bytes(int batch, int dim, int64_t seqlen);

/*
 * ssm_gated_scan_fwd -- the recurrence over whole sequences.
 *
 *   x, r         in   (batch, dim, seqlen), dtype       required
 *   A            in   (dim) float32                     required
 *   r_bias       in   (dim) float32                     NULL -> 0
 *   i            in   (batch, dim, seqlen), dtype       NULL -> no input gate
 *   i_bias       in   (dim) float32                     NULL -> 0; not read without i
 *   z            in   (batch, dim, seqlen), dtype       NULL -> no output gate
 *   flags        bits of ssm_gate_flag_t
 *   starts       in   (batch, seqlen) bytes             NULL -> none
 *   h0           in   (batch, dim) float32              NULL -> zero state
 *   y            out  (batch, dim, seqlen), dtype       required
 *   last_state   out  (batch, dim) float32              NULL -> not written
 *   ckpt         out  ssm_gated_scan_ckpt_bytes(...)    NULL -> not written
 *                     bytes or more (SSM_ERR_WORKSPACE), 4-byte aligned: what
 *                     ssm_gated_scan_bwd starts from
 *   batch, dim, seqlen >= 0; batch * dim at most 2^31 - 513, seqlen at most
 *   2^31 - 4097 (SSM_ERR_SHAPE); no workspace.  seqlen == 0 only
 *   writes last_state (= h0, or zeros).
 */
int ssm_gated_scan_fwd(const void* x, const void* r, const float* A, const float* r_bias,
                       const void* i, const float* i_bias, const void* z, int flags,
                       const uint8_t* starts, const float* h0, void* y, float* last_state,
                       float* ckpt, size_t ckpt_bytes, int batch, int dim, int64_t seqlen,
                       int dtype, void* stream);

/*
 * ssm_gated_scan_bwd -- gradients of a loss through ssm_gated_scan_fwd, given
 * dy and optionally the gradient of last_state.  With the adjoint
 * lambda_t = dy_t silu(z_t) + a_{t+1} lambda_{t+1} every gradient is the chain
 * rule through the formula at the top; the states are computed again from the
 * inputs, 512 steps at a time from the kept ones.
 *
 *   x .. starts  in   as for ssm_gated_scan_fwd (the same values)
 *   ckpt         in   what ssm_gated_scan_fwd wrote for them (its first entry
 *                     is h0)                                   required
 *   dy           in   (batch, dim, seqlen), dtype              required
 *   dlast_state  in   (batch, dim) float32                     NULL -> 0
 *   dx, dr       out  (batch, dim, seqlen), dtype              required
 *   dA           out  (dim) float32                            required
 *   dr_bias      out  (dim) float32                            NULL -> not written
 *   di           out  (batch, dim, seqlen), dtype              required when i is given
 *   di_bias      out  (dim) float32                            NULL -> not written; written
 *                                                              with i, and for an empty sequence
 *   dz           out  (batch, dim, seqlen), dtype              required when z is given
 *   dh0          out  (batch, dim) float32                     NULL -> not written
 *   workspace    at least ssm_gated_scan_bwd_workspace_bytes(...) bytes,
 *                256-byte aligned, owned by the caller (NULL where the query
 *                returns 0); calls sharing one workspace must not overlap
 * The sums over batch and steps have a fixed order.  batch == 0 or
 * seqlen == 0 writes zeros to dA and the bias gradients, and dh0 = dlast_state
 * (or zeros).
 */
int ssm_gated_scan_bwd(const void* x, const void* r, const float* A, const float* r_bias,
                       const void* i, const float* i_bias, const void* z, int flags,
                       const uint8_t* starts, const float* ckpt, size_t ckpt_bytes, const void* dy,
                       const float* dlast_state, void* dx, void* dr, float* dA, float* dr_bias,
                       void* di, float* di_bias, void* dz, float* dh0, int batch, int dim,
                       int64_t seqlen, int dtype, void* workspace, size_t workspace_bytes,
                       void* stream);

/* Bytes of device workspace of ssm_gated_scan_bwd.  Pure host function; 0 for
 * an empty problem and for arguments that it would refuse. */
size_t ssm_gated_scan_bwd_workspace_bytes(int batch, int dim, int64_t seqlen, int dtype);

/*
 * ssm_gated_state_update -- one token per sequence: the formula above with
 * seqlen = 1, from `state`.
 *
 *   state        in   (batch, dim) float32                     required;
 *                in/out where state_out is NULL or state itself
 *   x, r, i, z   in   (batch, dim), dtype                      as above
 *   starts       in   (batch) bytes: not 0 where the token is its sequence's
 *                     first                                    NULL -> none
 *   y            out  (batch, dim), dtype                      required
 *   state_out    out  (batch, dim) float32: the state after the token, where
 *                     the one before it is kept (a draft that may be taken
 *                     back)                                    NULL -> state
 */
int ssm_gated_state_update(float* state, const void* x, const void* r, const float* A,
                           const float* r_bias, const void* i, const float* i_bias, const void* z,
                           int flags, const uint8_t* starts, void* y, float* state_out, int batch,
                           int dim, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_GATED_H */
