/*
 * ssm_linear_attn.h -- C ABI of libssm: linear attention with a decay for each
 * head, its backward pass and its one-token step, on AMD Instinct MI355X (gfx950).
 *
 * The operation, for each batch row and head h of `heads` (S is a (key_dim,
 * value_dim) matrix):
 *
 *   S_t = exp(log_decay[h]) * S_{t-1} + k_t v_t^T      (S_{t-1} taken as 0 where starts[b,t] is not 0)
 *   y_t = scale * q_t S_t
 *
 * that is y_t = scale * sum over s <= t of exp(log_decay[h] (t-s)) (q_t . k_s) v_s:
 * attention without a softmax, its memory a state of constant size.  It is the
 * SSD form of ssm.h with keys and queries of each head's own (there B and C, shared
 * by all), a constant decay, and any head width.
 *
 * Conventions as in ssm.h (device pointers, stream, validation before any HIP
 * call, aliasing judged on byte ranges, deterministic results), and:
 *  - dtype (SSM_F32 or SSM_BF16) selects the storage of q, k, v, y and their
 *    gradients.  log_decay and the states are float32.
 *  - q: (batch, seqlen, q_heads, key_dim), k: (batch, seqlen, k_heads, key_dim),
 *    v: (batch, seqlen, v_heads, value_dim); y, dy: (batch, seqlen, heads,
 *    value_dim); states: (batch, heads, key_dim, value_dim).  q_heads, k_heads and
 *    v_heads each divide heads: head h reads head h / (heads / n) of n.
 *  - strides: a host array of 9, the elements from one batch row, step and head to
 *    the next of q, then of k, then of v (widths are contiguous): views of one
 *    projection's output are read where they lie.  NULL -> contiguous.  Not
 *    negative, at most 2^40, SSM_ERR_SHAPE otherwise.  Everything else is contiguous.
 *  - Pointers need their element's alignment only; where q, k or v is aligned to 16
 *    bytes with all its strides and its width it is read 16 bytes at a time, and 4
 *    where they are aligned to 4.
 *  - starts: (batch, seqlen) bytes, not 0 at the first step of each sequence
 *    packed into a row (a row may begin in the middle of one).  No state, no
 *    gradient and no NaN or Inf crosses a start.  NULL -> none.
 *  - lengths: (batch) int32, the steps of each row, a padded batch; values are
 *    taken into [0, seqlen].  What lies behind is not read; y and the gradients
 *    there are 0, and last_state is that of the row's last step (h0 where it has
 *    none).  NULL -> seqlen.
 *  - The state, the sums and the decays are held in float32; with bf16 storage the
 *    decayed products q_t . k_s as they meet v on the matrix cores, and the state as
 *    it meets q, are two bf16 parts (2^-16 of each, and what lies below 2^-126); in
 *    dlog_decay both are exact.
 *  - log_decay is not checked for sign; a positive one grows.  e^(64 log_decay), by
 *    itself and times the values of v, dy and q.k, has to be a float32: log_decay is at
 *    most 1.38, and 1.3 leaves room for values of 100 (above that, results may be NaN
 *    where the formula's are finite).  -inf forgets all but the step itself, of finite
 *    values.  A decay over many steps that underflows is held at the smallest normal
 *    float where log_decay > -87; a state that is not finite stays so until the next
 *    start, whatever the decay.
 *  - What a NaN or Inf reaches by the formula is not finite.  An Inf may be NaN there:
 *    the factors of a product are taken in parts, Inf - Inf one of them, and a value
 *    that is not finite makes the later y of its chunk NaN.  Earlier steps, sequences of
 *    their own, other heads and, of v, other columns are what they were.
 *    (dlog_decay is a sum over its head's whole rows: any of them may make it NaN.)
 */
#ifndef SSM_LINEAR_ATTN_H
#define SSM_LINEAR_ATTN_H

#include "ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Widest key_dim and value_dim. */
#define SSM_LINEAR_ATTN_MAX_DIM 256

/*
 * ssm_linear_attn_fwd -- whole sequences.
 *
 *   q, k, v      in   dtype                                    required
 *   strides      host array of 9                               NULL -> contiguous
 *   log_decay    in   (heads) float32                          required
 *   scale        finite (SSM_ERR_SHAPE otherwise)
 *   starts       in   (batch, seqlen) bytes                    NULL -> none
 *   lengths      in   (batch) int32                            NULL -> seqlen
 *   h0           in   (batch, heads, key_dim, value_dim)       NULL -> zero state
 *   y            out  (batch, seqlen, heads, value_dim)        required
 *   last_state   out  as h0                                    NULL -> not written
 *   workspace    at least ssm_linear_attn_fwd_workspace_bytes(...) bytes,
 *                256-byte aligned, owned by the caller (NULL where the query
 *                returns 0); calls sharing one workspace must not overlap
 *   batch, seqlen, heads >= 0; q_heads, k_heads, v_heads >= 1 and dividing heads;
 *   key_dim and value_dim 1 to 256; seqlen at most 2^31 - 4097, batch * heads at
 *   most 2^31 - 4097 (SSM_ERR_SHAPE).  seqlen == 0 only writes last_state.
 */
int ssm_linear_attn_fwd(const void* q, const void* k, const void* v, const int64_t* strides,
                        const float* log_decay, float scale, const uint8_t* starts,
                        const int32_t* lengths, const float* h0, void* y, float* last_state,
                        int batch, int64_t seqlen, int heads, int q_heads, int k_heads, int v_heads,
                        int key_dim, int value_dim, int dtype, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Bytes of device workspace of ssm_linear_attn_fwd (states entering the parts
 * that long rows are split into).  Pure host function; 0 for an empty problem and
 * for arguments that it would refuse. */
size_t ssm_linear_attn_fwd_workspace_bytes(int batch, int64_t seqlen, int heads, int key_dim,
                                           int value_dim, int dtype);

/*
 * ssm_linear_attn_bwd -- gradients of a loss through ssm_linear_attn_fwd, given dy
 * and optionally the gradient of last_state:
 *
 *   dS_t = scale q_t^T dy_t + exp(log_decay) dS_{t+1}   (dS_{t+1} = 0 where t+1 starts a sequence)
 *   dq_t = scale S_t dy_t,   dk_t = dS_t v_t,   dv_t = dS_t^T k_t
 *   dlog_decay = sum over batch and t of <dS_t, exp(log_decay) S_{t-1}>
 *
 *   q .. h0      in   as for ssm_linear_attn_fwd (the same values)
 *   dy           in   (batch, seqlen, heads, value_dim), dtype  required
 *   dlast_state  in   as h0                                     NULL -> 0
 *   dq, dk, dv   out  contiguous, in the shapes of q, k, v; heads that share
 *                     one are summed in a fixed order           required
 *   dlog_decay   out  (heads) float32                           NULL -> not computed
 *   dh0          out  as h0                                     NULL -> not written
 *   workspace    as above, of ssm_linear_attn_bwd_workspace_bytes(...)
 * batch == 0 or seqlen == 0 writes zeros to dlog_decay, and dh0 = dlast_state (or
 * zeros).
 */
int ssm_linear_attn_bwd(const void* q, const void* k, const void* v, const int64_t* strides,
                        const float* log_decay, float scale, const uint8_t* starts,
                        const int32_t* lengths, const float* h0, const void* dy,
                        const float* dlast_state, void* dq, void* dk, void* dv, float* dlog_decay,
                        float* dh0, int batch, int64_t seqlen, int heads, int q_heads, int k_heads,
                        int v_heads, int key_dim, int value_dim, int dtype, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Bytes of device workspace of ssm_linear_attn_bwd.  Pure host function; 0 for an
 * empty problem and for arguments that it would refuse. */
size_t ssm_linear_attn_bwd_workspace_bytes(int batch, int64_t seqlen, int heads, int q_heads,
                                           int k_heads, int v_heads, int key_dim, int value_dim,
                                           int dtype);

/*
 * ssm_linear_attn_state_update -- one token per sequence: the formula above with
 * seqlen = 1, from `state`.
 *
 *   state        in   (batch, heads, key_dim, value_dim) float32  required;
 *                in/out where state_out is NULL or state itself
 *   q, k, v      in   (batch, n heads, width), dtype              required
 *   strides      host array of 6: batch and head of q, k, v       NULL -> contiguous
 *   starts       in   (batch) bytes: not 0 where the token is its sequence's
 *                     first                                       NULL -> none
 *   y            out  (batch, heads, value_dim), dtype            required
 *   state_out    out  as state: the state after the token, where the one before
 *                     it is kept (a draft that may be taken back) NULL -> state
 */
int ssm_linear_attn_state_update(float* state, const void* q, const void* k, const void* v,
                                 const int64_t* strides, const float* log_decay, float scale,
                                 const uint8_t* starts, void* y, float* state_out, int batch,
                                 int heads, int q_heads, int k_heads, int v_heads, int key_dim,
                                 int value_dim, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_LINEAR_ATTN_H */
