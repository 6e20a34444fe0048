// gated_math.hpp -- the gated recurrence's per-element arithmetic and its
// composition over a wave (gfx950).  include/ssm_gated.h states the formula.
#pragma once

#include "runs.hpp"

namespace ssm {

// Rules of the gate and of the input weight (bits of the RULE argument).
constexpr int kGateSoftplus = 1;
constexpr int kGateUnit = 2;

// sigmoid(x) = 1/(1 + e^-x): 0 at -inf, where e^-x is infinite.
__device__ __forceinline__ float sigmoid_f32(float x) { return rcp_hw(1.0f + exp2_hw(-x * kLog2e)); }

// sigmoid(x) and 1 - sigmoid(x) = e^-x sigmoid(x), the latter without
// cancellation.  Where e^-x is infinite the product 0 * inf is NaN and the
// minimum returns its other operand, 1.
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& c) {
  const float t = exp2_hw(-x * kLog2e);
  s = rcp_hw(1.0f + t);
  c = __builtin_fminf(t * s, 1.0f);
}

// 1 - e^t for t <= 0 (any t works): where |t| < 1/4 the difference would
// magnify the rounding of e^t, so the Taylor series -t (1 + t/2 + ... +
// t^5/720) is taken (dropped terms below t^6/5040 < 5e-8 relative), elsewhere
// 1 - e^t with `et` = e^t.  Branch-free.  A NaN t takes the series, and stays
// NaN whatever `et` is.
__device__ __forceinline__ float one_minus_exp(float t, float et) {
  float p = __builtin_fmaf(t, 1.0f / 720.0f, 1.0f / 120.0f);
  p = __builtin_fmaf(t, p, 1.0f / 24.0f);
  p = __builtin_fmaf(t, p, 1.0f / 6.0f);
  p = __builtin_fmaf(t, p, 0.5f);
  p = __builtin_fmaf(t, p, 1.0f);
  return __builtin_fabsf(t) >= 0.25f ? 1.0f - et : -t * p;
}

// The decay of one step from its base-2 exponent e2 = A log2(e) g, held at or
// above the smallest normal float: exp is never 0, and an infinite state that
// met a decay flushed to 0 would turn into NaN.  (A NaN exponent gives the
// floor here; the input weight of that step is NaN and reaches the state.)
__device__ __forceinline__ float decay_of(float e2) { return __builtin_fmaxf(exp2_hw(e2), kMinNormal); }

// The input weight: 1 - a, or sqrt(1 - a^2) = sqrt(1 - e^(2 A g)); An = A or
// 2A accordingly, so that An * g is the exponent whose complement is taken.
template <int RULE>
__device__ __forceinline__ float weight_of(float a, float An, float g) {
  if constexpr ((RULE & kGateUnit) != 0) {
    return __builtin_amdgcn_sqrtf(one_minus_exp(An * g, a * a));
  } else {
    return one_minus_exp(An * g, a);
  }
}

// Bit k set where a sequence starts at step k of the run.
__device__ __forceinline__ uint32_t load_starts(const uint8_t* p, int valid) {
  typedef uint32_t vec2 __attribute__((ext_vector_type(2), aligned(1)));
  uint32_t m = 0;
  if (valid >= kRun) {
    const vec2 v = *reinterpret_cast<const vec2*>(p);
#pragma unroll
    for (int k = 0; k < kRun; ++k) m |= (((k < 4 ? v.x : v.y) >> (8 * (k & 3))) & 0xffu) != 0 ? 1u << k : 0u;
  } else {
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      if (k < valid && p[k] != 0) m |= 1u << k;
  }
  return m;
}

// ---- composition over the wave -------------------------------------------------
// A run of steps is the map h -> P h + Q.  P = 0 marks a run holding a start:
// it forgets h whatever h is (0 * inf is not formed); every other P is at or
// above the smallest normal float.  CUT false: no starts, P is never 0.
template <bool CUT>
__device__ __forceinline__ float apply_map(float P, float Q, float h) {
  const float v = __builtin_fmaf(P, h, Q);
  return CUT && P == 0.0f ? Q : v;
}

// (P, Q) after (Pf, Qf).
template <bool CUT>
__device__ __forceinline__ void compose_map(float& P, float& Q, float Pf, float Qf) {
  Q = apply_map<CUT>(P, Q, Qf);
  const float pp = __builtin_fmaxf(P * Pf, kMinNormal);
  P = CUT && (P == 0.0f || Pf == 0.0f) ? 0.0f : pp;
}

// One round of the inclusive prefix: lanes that the DPP control names a source
// for compose their map after that lane's, the others keep theirs.
template <bool CUT, int CTRL, int ROW_MASK>
__device__ __forceinline__ void prefix_round(float& P, float& Q) {
  const float qf =
      __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(Q), CTRL, ROW_MASK, 0xf, false));
  const float pf = __int_as_float(
      __builtin_amdgcn_update_dpp(__float_as_int(1.0f), __float_as_int(P), CTRL, ROW_MASK, 0xf, false));
  compose_map<CUT>(P, Q, pf, qf);
}

// Inclusive prefix of the lanes' maps, lane 0 first.
template <bool CUT>
__device__ __forceinline__ void wave_prefix(float& P, float& Q) {
  prefix_round<CUT, 0x111, 0xf>(P, Q);  // row_shr:1
  prefix_round<CUT, 0x112, 0xf>(P, Q);  // row_shr:2
  prefix_round<CUT, 0x114, 0xf>(P, Q);  // row_shr:4
  prefix_round<CUT, 0x118, 0xf>(P, Q);  // row_shr:8
  prefix_round<CUT, 0x142, 0xa>(P, Q);  // row_bcast:15 into rows 1 and 3
  prefix_round<CUT, 0x143, 0xc>(P, Q);  // row_bcast:31 into rows 2 and 3
}

// The value of the lane before (`first` in lane 0).
__device__ __forceinline__ float lane_before(float v, float first) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(first), __float_as_int(v), 0x138, 0xf, 0xf, false));
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// The value of lane 63 - lane.
__device__ __forceinline__ float lane_mirror(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_ds_bpermute((63 - lane) * 4, __float_as_int(v)));
}

}  // namespace ssm
