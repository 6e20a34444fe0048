// runs.hpp -- vector accesses to runs of consecutive elements at any alignment
// (gfx950), and sums over a wave.
#pragma once

#include <type_traits>

#include "ssm_math.hpp"

namespace ssm {

constexpr int kRun = 8;  // consecutive elements that a lane holds

// A grid of `groups` workgroups or a few more.  A dimension of a grid has fewer
// than 2^32 threads: past 2^31 the workgroups go to a second one.
inline dim3 grid_of(int64_t groups, int threads) {
  const int64_t most = (INT64_C(1) << 31) / threads, y = (groups + most - 1) / most;
  return dim3((unsigned)((groups + y - 1) / y), (unsigned)y);
}

// The workgroup's number in such a grid.
__device__ __forceinline__ int64_t group_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// ---- runs of kRun consecutive elements of a row --------------------------------
// Rows start at any element (their length need not be a multiple of the run), so the
// vector accesses are declared with the element's alignment; global memory
// takes them at any byte address on gfx950.
typedef uint32_t vec4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t vec4_at4 __attribute__((ext_vector_type(4), aligned(4)));

template <typename T>
struct RunWords {
  typedef typename std::conditional<sizeof(T) == 2, vec4_at2, vec4_at4>::type vec4;
  static constexpr int kWords = kRun * (int)sizeof(T) / 4;
  uint32_t w[kWords];
};

// Elements p[0 .. kRun-1]; those from `valid` on read as zero and are not
// touched.  ONCE: read past the caches (non-temporal).
template <typename T, bool ONCE = false>
__device__ __forceinline__ RunWords<T> load_run(const T* p, int valid) {
  typedef typename RunWords<T>::vec4 vec4;
  RunWords<T> r;
  if (valid >= kRun) {
#pragma unroll
    for (int q = 0; q < RunWords<T>::kWords / 4; ++q) {
      const vec4 v = ONCE ? __builtin_nontemporal_load(reinterpret_cast<const vec4*>(p) + q)
                          : reinterpret_cast<const vec4*>(p)[q];
      r.w[4 * q] = v.x; r.w[4 * q + 1] = v.y; r.w[4 * q + 2] = v.z; r.w[4 * q + 3] = v.w;
    }
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int q = 0; q < kRun / 2; ++q) {
      const uint32_t lo = 2 * q < valid ? (uint32_t)p[2 * q] : 0u;
      const uint32_t hi = 2 * q + 1 < valid ? (uint32_t)p[2 * q + 1] : 0u;
      r.w[q] = lo | (hi << 16);
    }
  } else {
#pragma unroll
    for (int q = 0; q < kRun; ++q) r.w[q] = q < valid ? __float_as_uint(p[q]) : 0u;
  }
  return r;
}

// Store the first `valid` of kRun floats as T (bf16: round to nearest even).
// ONCE: as above.
template <typename T, bool ONCE = false>
__device__ __forceinline__ void store_run(T* p, int valid, const float (&f)[kRun]) {
  typedef typename RunWords<T>::vec4 vec4;
  if (valid >= kRun) {
    uint32_t w[RunWords<T>::kWords];
    pack_floats<T, kRun>(f, w);
#pragma unroll
    for (int q = 0; q < RunWords<T>::kWords / 4; ++q) {
      const vec4 v = {w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]};
      if constexpr (ONCE) __builtin_nontemporal_store(v, reinterpret_cast<vec4*>(p) + q);
      else reinterpret_cast<vec4*>(p)[q] = v;
    }
  } else {
#pragma unroll
    for (int q = 0; q < kRun; ++q)
      if (q < valid) Elem<T>::store(p + q, f[q]);
  }
}

template <typename T>
__device__ __forceinline__ void run_floats(const RunWords<T>& r, float (&f)[kRun]) {
  words_to_floats<T, kRun>(r.w, f);
}

// A float64 by two moves of its halves.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_moved(double v) {
  return __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, ROW_MASK, 0xf, false),
                          __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, ROW_MASK, 0xf, false));
}

__device__ __forceinline__ float last_lane(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double last_lane(double v) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), 63),
                          __builtin_amdgcn_readlane(__double2loint(v), 63));
}

// The sum of v over the wave, in every lane; the order is fixed.
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
  v += dpp_moved<0x111, 0xf>(v);  // row_shr:1
  v += dpp_moved<0x112, 0xf>(v);  // row_shr:2
  v += dpp_moved<0x114, 0xf>(v);  // row_shr:4
  v += dpp_moved<0x118, 0xf>(v);  // row_shr:8
  v += dpp_moved<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v += dpp_moved<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  return last_lane(v);
}

}  // namespace ssm
