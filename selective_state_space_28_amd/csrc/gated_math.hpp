// gated_math.hpp -- the gated recurrence's per-element arithmetic and its
// composition over a wave (gfx950).  include/ssm_gated.h states the formula.
#pragma once

#include "runs.hpp"

namespace ssm {

// Rules of the gate and of the input weight (bits of the RULE argument).
constexpr int kGateSoftplus = 1;
constexpr int kGateUnit = 2;

// sigmoid(x + bias) = 1/(1 + e^-(x + bias)), with nb = -bias log2(e): 0 at -inf,
// where the exponential is infinite.
__device__ __forceinline__ float sigmoid_f32(float x, float nb) {
  return rcp_hw(1.0f + exp2_hw(__builtin_fmaf(x, -kLog2e, nb)));
}

// The same and its complement e^-x sigmoid(x), the latter without cancellation.
// Where e^-x is infinite the product 0 * inf is NaN and the minimum returns its
// other operand, 1.
__device__ __forceinline__ void sigmoid_pair(float x, float nb, float& s, float& c) {
  const float t = exp2_hw(__builtin_fmaf(x, -kLog2e, nb));
  s = rcp_hw(1.0f + t);
  c = __builtin_fminf(t * s, 1.0f);
}

// softplus(x) and its slope sigmoid(x) from one exponential: with w = e^-|x| the
// slope is 1/(1 + w) or w/(1 + w).
__device__ __forceinline__ void softplus_pair(float x, float& sp, float& slope) {
  const float w = exp2_hw(-__builtin_fabsf(x) * kLog2e);
  sp = __int_as_float(max(__float_as_int(x), 0)) + log1p_unit(w);
  slope = rcp_hw(1.0f + w) * (x < 0.0f ? w : 1.0f);
}

// The gate of one step: its value g, the base-2 exponent e2 = A log2(e) g of the
// decay, the decay a and the input weight w.
//
// The decay is held at or above the smallest normal float: exp is never 0, and an
// infinite state that met a decay flushed to 0 would turn into NaN.  A NaN
// exponent gives a NaN decay (the maximum that keeps it; a run's is floored
// all the same, and the run's Q carries the NaN): the backward pass' adjoint
// has it to itself, where the state has the step's weight too.
//
// The weight is 1 - e^t, or its root, with t = A g or 2 A g.  Where |t| < 1/8 the
// difference would magnify the rounding of e^t, so -t (e^t - 1)/t is taken, the
// quotient as the cubic through its values at the Chebyshev nodes of [-1/8, 1/8]
// (2.7e-7 relative at most), in powers of e2; elsewhere the difference itself,
// whose rounding is then 2^-24 / 0.118 = 5e-7 relative at most.  Branch-free; a
// NaN takes the cubic and stays NaN.
struct Gate {
  float g, e2, a, w;
};

template <int RULE>
__device__ __forceinline__ Gate gate_of(float g, float A2) {
  constexpr bool unit = (RULE & kGateUnit) != 0;
  constexpr float s = unit ? 2.0f * kLn2 : kLn2;  // t = s e2
  constexpr float k0 = -0.99999974559f * s, k1 = -0.49999995760f * s * s, k2 = -0.16679691739f * s * s * s,
                  k3 = -0.04168837335f * s * s * s * s;
  Gate r;
  r.g = g;
  r.e2 = A2 * g;
  r.a = __builtin_elementwise_maximum(exp2_hw(r.e2), kMinNormal);
  float p = __builtin_fmaf(r.e2, k3, k2);
  p = __builtin_fmaf(r.e2, p, k1);
  p = __builtin_fmaf(r.e2, p, k0);
  const float far = unit ? __builtin_fmaf(-r.a, r.a, 1.0f) : 1.0f - r.a;
  const float m = __builtin_fabsf(r.e2) >= 0.125f / s ? far : r.e2 * p;
  r.w = unit ? __builtin_amdgcn_sqrtf(m) : m;
  return r;
}

// Bit k set where a sequence starts at step k of a run of N (8 or 4).
template <int N>
__device__ __forceinline__ uint32_t load_starts(const uint8_t* p, int valid) {
  typedef uint32_t vec2 __attribute__((ext_vector_type(2), aligned(1)));
  typedef uint32_t word __attribute__((aligned(1)));
  uint32_t m = 0;
  if (valid >= N) {
    uint32_t w[2] = {0u, 0u};
    if constexpr (N == 8) {
      const vec2 v = *reinterpret_cast<const vec2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const word*>(p);
    }
    // (a bare "no start in the run" is the common answer)
    if ((w[0] | w[1]) != 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) m |= ((w[k / 4] >> (8 * (k & 3))) & 0xffu) != 0 ? 1u << k : 0u;
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
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
  if constexpr (CUT) {
    prefix_round<CUT, 0x111, 0xf>(P, Q);  // row_shr:1
    prefix_round<CUT, 0x112, 0xf>(P, Q);  // row_shr:2
    prefix_round<CUT, 0x114, 0xf>(P, Q);  // row_shr:4
    prefix_round<CUT, 0x118, 0xf>(P, Q);  // row_shr:8
    prefix_round<CUT, 0x142, 0xa>(P, Q);  // row_bcast:15 into rows 1 and 3
    prefix_round<CUT, 0x143, 0xc>(P, Q);  // row_bcast:31 into rows 2 and 3
  } else {
    // The same rounds without starts, the lane shift in the operation itself:
    // Q += P Q_from, P = max(P P_from, the smallest normal float); a lane without
    // a source is not written and keeps its map.  (From the compiler each shift
    // is a move of its own: 5 instructions a round instead of 3.)  An operand
    // that comes from another lane must have been written two instructions
    // before: the waits stand for those that are missing.
#define SSM_ROUND(SHIFT)                             \
  "v_fmac_f32_dpp %1, %1, %0 " SHIFT " bank_mask:0xf\n" \
  "s_nop 0\n"                                        \
  "v_mul_f32_dpp %0, %0, %0 " SHIFT " bank_mask:0xf\n"  \
  "v_max_f32_e32 %0, 0x800000, %0\n"
    asm("s_nop 1\n"
        SSM_ROUND("row_shr:1 row_mask:0xf")
        SSM_ROUND("row_shr:2 row_mask:0xf")
        SSM_ROUND("row_shr:4 row_mask:0xf")
        SSM_ROUND("row_shr:8 row_mask:0xf")
        SSM_ROUND("row_bcast:15 row_mask:0xa")
        SSM_ROUND("row_bcast:31 row_mask:0xc")
        "s_nop 1"
        : "+v"(P), "+v"(Q));
#undef SSM_ROUND
  }
}

// The value of the lane before (`first` in lane 0).
__device__ __forceinline__ float lane_before(float v, float first) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(first), __float_as_int(v), 0x138, 0xf, 0xf, false));
}

// The value of the lane after (`last` in lane 63).
__device__ __forceinline__ float lane_after(float v, float last) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(last), __float_as_int(v), 0x130, 0xf, 0xf, false));
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// The value of lane 63 - lane.
__device__ __forceinline__ float lane_mirror(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_ds_bpermute((63 - lane) * 4, __float_as_int(v)));
}

}  // namespace ssm
