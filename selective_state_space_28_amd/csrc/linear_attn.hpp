// linear_attn.hpp -- what a sweep of the linear attention takes (linear_attn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm_kernels.hpp"

namespace ssm {

constexpr int kAttnMaxWidth = 256;  // widest key or value head
constexpr int kAttnChunk = 64;      // steps of a chunk with 16-bit operands; segments are multiples of it

// A (batch, step, head, width) operand: strides in elements, the width's is 1;
// head h of the recurrence reads head h / share.
struct AttnView {
  const void* p;
  int64_t sb, st, sh;
  int share;
};

// One sweep of the chunked recurrence over the steps of every row,
//   S_u = e^g S_{u-1} + scale_upd k_u v_u^T,   out_u = q_u . S
// in the order of the steps or, `rev`, from the last to the first.  Every pass of
// the operator is one with its operands in other places (linear_attn.hip).
struct AttnSweep {
  AttnView q, k, v;   // q, k: kd wide; v: vd wide
  AttnView dy;        // the decay's gradient only
  void* out;          // (batch, seqlen, heads, vd), dtype, or float32 (out_f32)
  int out_f32;
  int kd, vd, batch, heads;
  int64_t seqlen;
  const float* g;          // (heads) log decay of a step
  float scale_p, scale_in, scale_upd;
  const uint8_t* starts;   // nullable
  const int32_t* lengths;  // nullable
  int rev;
  const float* state_in;   // nullable; (batch, heads, kd, vd), or (vd, kd) if transposed
  float* state_out;        // nullable
  int transposed;
  float* seg_state;   // (batch, heads, nseg, kd, vd): states entering the segments, when nseg > 1
  float* seg_rate;    // the decay's gradient only: its derivative by g, as seg_state
  float* seg_steps;   // and the steps of the segments, as seg_through
  float* seg_through; // (batch, heads, nseg): what a segment leaves of the state that enters it (through_of)
  int64_t seglen;     // steps of a segment, a multiple of kAttnChunk
  int nseg;
  double* part;       // decay's gradient: (heads, batch, column blocks, nseg)
  Dtype dtype;
};

// Sweeps that run side by side: of the same sizes but for kd and vd, which are alike
// (attn_alike), and with the same segments.
struct AttnSweeps {
  AttnSweep s[3];
  int n;
};
bool attn_alike(int a, int b);

// Segments that `groups` (sweeps, batch rows, heads and blocks of value columns) of
// seqlen steps, with so many elements in their states, are split into, and their steps.
struct AttnSplit {
  int nseg;
  int64_t seglen;
};
AttnSplit attn_split(int64_t groups, int64_t seqlen, int64_t state_elements, Dtype dtype);
// Blocks of value columns, of a sweep and of the decay's gradient.
int attn_column_blocks(int vd);
int attn_decay_blocks(int vd);

struct AttnStep {
  AttnView q, k, v;  // (batch, head, width): st is not used
  const float* g;
  float scale;
  const uint8_t* starts;  // nullable
  const float* state;
  float* state_out;
  void* y;
  int batch, heads, kd, vd;
  Dtype dtype;
};

hipError_t launch_attn_sweeps(const AttnSweeps& all, hipStream_t stream);
// dlog_decay (heads): the sum over batch and steps; a.q, a.k, a.v as in the forward sweep, a.dy the gradient of its
// output, dlast that of its last state (nullable).
hipError_t launch_attn_decay_grad(const AttnSweep& a, const float* dlast, float* dlog_decay, hipStream_t stream);
// out (batch, seqlen, n, width) of part (batch, seqlen, heads, width): the sum over the heads / n that share a head.
hipError_t launch_attn_gather(const float* part, void* out, int64_t rows, int heads, int n, int width, Dtype dtype,
                              hipStream_t stream);
hipError_t launch_attn_step(const AttnStep& a, hipStream_t stream);

}  // namespace ssm
