// group_norm.hip -- the norm of groups of a token's channels with an activation or
// a gate, forward and backward, for gfx950 (include/ssm_group_norm.h states it).
//
// Both directions are bound by HBM: some 13 and 28 operations an element against 6
// to 10 bytes of bf16.  A group lies in the registers of 1 to 64 lanes of a wave, or
// of a workgroup of 256 (groups of more than 1024 channels), each kRun channels K
// times, so it is read once; its sums go over the lanes by DPP.  A wave keeps its
// channels and goes over tokens, so that weight and bias are read once, and the
// sums of dweight and dbias stay in registers until its last token.  32768 tokens of 5120
// bf16 in groups of 128 with a gate: 197 us, 5.2 TB/s; the backward of half of them 175, 4.8.
#include <algorithm>

#include "gated_math.hpp"
#include "runs.hpp"
#include "ssm_group_norm.h"
#include "ssm_kernels.hpp"

namespace ssm {

namespace {

constexpr int kWaves = 4;    // of a workgroup
constexpr int kBlockSpan = 64 * kWaves;

// Workgroups that share the tokens.  Forward: many, a few tokens a wave (32768 tokens of
// 5120 bf16 in groups of 128, with a gate: 191 us; with 2048 of them 234, with 32768
// 217).  Backward: each leaves a part of dweight and dbias, so fewer, with 32 tokens to a
// part where that leaves 512 (16384 tokens of 5120: 177 us; with 1024 of them 185; but
// 4096 tokens of 8192 in one group: 124 us with 1024, 173 with 2048, 260 with 4096).
// Loading a token ahead cost both (191 -> 200, 176 -> 191).
constexpr int kFwdGroups = 8192, kBwdGroups = 2048, kBwdLeast = 512, kPartTokens = 32;

// Sum over the LR lanes of a group, in every lane of it; the order is fixed.
template <int LR, typename V>
__device__ __forceinline__ V group_sum(V v, V* s) {
  if constexpr (LR >= 2) v += dpp_moved<0xb1, 0xf>(v);   // quad_perm: the pair's other
  if constexpr (LR >= 4) v += dpp_moved<0x4e, 0xf>(v);   // quad_perm: the other pair
  if constexpr (LR >= 8) v += dpp_moved<0x141, 0xf>(v);  // row_half_mirror: the other 4 of 8
  if constexpr (LR >= 16) v += dpp_moved<0x140, 0xf>(v);  // row_mirror: the other 8 of 16
  if constexpr (LR >= 32) v += __shfl_xor(v, 16);
  if constexpr (LR >= 64) v += __shfl_xor(v, 32);
  if constexpr (LR > 64) {
    __syncthreads();  // the sum before has been read
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (s[0] + s[1]) + (s[2] + s[3]);
  }
  return v;
}

// What a group's values are summed in: exact for equal values (float32: float64,
// bf16: up to 2^16 values of 8 bits), and inside the type's range.
template <typename T>
using GroupSum = typename std::conditional<sizeof(T) == 4, double, float>::type;
constexpr float kSumScale = 1.0f / 65536;

// Groups whose squares pass float32's range (a part of a group at the type's lowest value, as
// masks have it) are taken again with deviations scaled by kFar: of up to 2^129, their squares
// sum to less than 2^112; of those whose squares passed 2^128 some exceed 2^57, 2^-23 scaled.
// The backward scales by kFarBack where rstd is below kFarRstd: deviations that pass the
// range have one below 2^-121, which may be subnormal; its product with 1 / kFarBack is exact.
constexpr float kFar = 0x1p-80f, kFarBack = 0x1p-24f, kFarRstd = 0x1p-100f, kMostFloat = 3.4028234664e38f;

__device__ __forceinline__ void load_par(const float* p, int valid, float otherwise, float (&f)[kRun]) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < kRun; ++k) f[k] = otherwise;
  } else {
    run_floats<float>(load_run<float>(p, valid), f);
  }
}

// The activation of t and, as `slope`, its derivative.
__device__ __forceinline__ float act_of(int act, float t, float& slope) {
  if (act == SSM_ACT_NONE) {
    slope = 1.0f;
    return t;
  }
  float s, c;
  sigmoid_pair(t, 0.0f, s, c);
  if (act == SSM_ACT_SIGMOID) {
    slope = s * c;
    return s;
  }
  slope = s * __builtin_fmaf(t, c, 1.0f);
  return t * s;
}

// A lane's place: `token` is its first, `step` the tokens to its next.
struct GroupPlace {
  int64_t token, step;
  int group, lane;  // group of the token, lane of the group
  bool live;
  int sub, per;     // token of the wave's `per` side by side, lanes of a token
};

template <int LR>
__device__ __forceinline__ GroupPlace group_place(int groups, int slabs, int64_t slices) {
  constexpr int kTeam = LR > 64 ? LR : 64;
  const int64_t id = group_index();
  const int slab = (int)(id % slabs);
  const int64_t slice = id / slabs;
  const int64_t lanes = (int64_t)groups * LR;  // of a token
  const int in_team = threadIdx.x % kTeam, wave = LR > 64 ? 0 : threadIdx.x / 64;
  constexpr int kTeams = kBlockSpan / kTeam;
  GroupPlace p;
  if (lanes < kTeam) {
    p.per = kTeam / (int)lanes;
    p.sub = in_team / (int)lanes;
    const int l = in_team - p.sub * (int)lanes;
    p.group = l / LR;
    p.lane = l % LR;
    p.live = p.sub < p.per;
  } else {
    const int64_t l = (int64_t)slab * kTeam + in_team;
    p.per = 1;
    p.sub = 0;
    p.group = (int)(l / LR);
    p.lane = (int)(l % LR);
    p.live = l < lanes;
  }
  p.token = (slice * kTeams + wave) * p.per + p.sub;
  p.step = slices * kTeams * p.per;
  return p;
}

}  // namespace

template <typename T, int K, int LR>
__global__ __launch_bounds__(kBlockSpan) void group_norm_fwd_kernel(const GroupNormLaunch a, int slabs, int64_t slices) {
  if (group_index() >= slabs * slices) return;
  __shared__ GroupSum<T> s_mean[kWaves];
  __shared__ float s_var[kWaves];
  const GroupPlace p = group_place<LR>(a.groups, slabs, slices);
  const int width = a.width;
  const int64_t c0 = (int64_t)p.group * width;
  float w[K][kRun], bias[K][kRun];
  int valid[K], at[K];
#pragma unroll
  for (int c = 0; c < K; ++c) {
    at[c] = (c * LR + p.lane) * kRun;
    valid[c] = p.live ? width - at[c] : 0;
    load_par(a.weight ? a.weight + c0 + at[c] : nullptr, valid[c], 1.0f, w[c]);
    load_par(a.bias ? a.bias + c0 + at[c] : nullptr, valid[c], 0.0f, bias[c]);
  }
  const T* x = static_cast<const T*>(a.x) + c0;
  const T* z = a.z == nullptr ? nullptr : static_cast<const T*>(a.z) + c0;
  T* y = static_cast<T*>(a.y) + c0;
  const float n = (float)width;
  const double rn = 1.0 / (double)width;
  for (int64_t t = p.token; t < a.tokens; t += p.step) {
    if (!p.live) break;
    float v[K][kRun];
    RunWords<T> zw[K];
    GroupSum<T> sum = 0;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      run_floats<T>(load_run(x + t * a.x_stride + at[c], valid[c]), v[c]);
      if (z != nullptr) zw[c] = load_run(z + t * a.z_stride + at[c], valid[c]);  // on its way with x
    }
#pragma unroll
    for (int c = 0; c < K; ++c) {
#pragma unroll
      for (int k = 0; k < kRun; ++k) sum = sizeof(T) == 4 ? sum + v[c][k] : __builtin_fmaf(v[c][k], kSumScale, sum);
    }
    sum = group_sum<LR>(sum, s_mean);
    const float mean = sizeof(T) == 4 ? (float)(sum * rn) : (float)sum / n * (1.0f / kSumScale);
    // the sum of the squares of the deviations, formed again for each use: v * scale - m
    float scale = 1.0f, m = mean;
    const auto sum_of_squares = [&] {
      float sq = 0.0f;
#pragma unroll
      for (int c = 0; c < K; ++c)
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          const float d = __builtin_fmaf(v[c][k], scale, -m);
          sq += k < valid[c] ? d * d : 0.0f;
        }
      return group_sum<LR>(sq, s_var);
    };
    float squares = sum_of_squares();
    if (!(squares <= kMostFloat)) {  // (alike in all lanes of the group)
      scale = kFar;
      m = mean * kFar;
      squares = sum_of_squares();
    }
    const float rstd = 1.0f / __builtin_sqrtf(squares / n + a.eps * scale * scale);  // of the scaled deviations
    if (p.lane == 0) {
      if (a.mean != nullptr) a.mean[t * a.groups + p.group] = mean;
      if (a.rstd != nullptr) a.rstd[t * a.groups + p.group] = rstd * scale;
    }
#pragma unroll
    for (int c = 0; c < K; ++c) {
      float f[kRun], slope;
      if (z != nullptr) run_floats<T>(zw[c], f);
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const float u = __builtin_fmaf(__builtin_fmaf(v[c][k], scale, -m) * rstd, w[c][k], bias[c][k]);
        f[k] = z != nullptr ? u * act_of(a.act, f[k], slope) : act_of(a.act, u, slope);
      }
      store_run<T, sizeof(T) == 2>(y + t * a.dim + at[c], valid[c], f);
    }
  }
}

template <typename T, int K, int LR>
__global__ __launch_bounds__(kBlockSpan) void group_norm_bwd_kernel(const GroupNormLaunch a, int slabs, int64_t slices) {
  if (group_index() >= slabs * slices) return;
  __shared__ float s_sum[2][kWaves];
  __shared__ float s_acc[LR > 64 ? 1 : kWaves - 1][64][kRun + 1];
  const GroupPlace p = group_place<LR>(a.groups, slabs, slices);
  const int width = a.width;
  const int64_t c0 = (int64_t)p.group * width;
  float w[K][kRun], bias[K][kRun], dw[K][kRun], db[K][kRun];
  int valid[K], at[K];
#pragma unroll
  for (int c = 0; c < K; ++c) {
    at[c] = (c * LR + p.lane) * kRun;
    valid[c] = p.live ? width - at[c] : 0;
    load_par(a.weight ? a.weight + c0 + at[c] : nullptr, valid[c], 1.0f, w[c]);
    load_par(a.bias ? a.bias + c0 + at[c] : nullptr, valid[c], 0.0f, bias[c]);
#pragma unroll
    for (int k = 0; k < kRun; ++k) dw[c][k] = db[c][k] = 0.0f;
  }
  const T* x = static_cast<const T*>(a.x) + c0;
  const T* z = a.z == nullptr ? nullptr : static_cast<const T*>(a.z) + c0;
  const T* dy = static_cast<const T*>(a.dy) + c0;
  T* dx = static_cast<T*>(a.dx) + c0;
  T* dz = static_cast<T*>(a.dz) + c0;
  const float rn = 1.0f / (float)width;
  for (int64_t t = p.token; t < a.tokens; t += p.step) {
    if (!p.live) break;
    const float mean = a.mean[t * a.groups + p.group], rstd = a.rstd[t * a.groups + p.group];
    const bool far = rstd < kFarRstd;
    const float scale = far ? kFarBack : 1.0f, m = mean * scale, r = far ? rstd * (1.0f / kFarBack) : rstd;
    float xh[K][kRun], d[K][kRun];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      float f[kRun];
      run_floats<T>(load_run(x + t * a.x_stride + at[c], valid[c]), xh[c]);
      run_floats<T>(load_run(dy + t * a.dim + at[c], valid[c]), d[c]);
      if (z != nullptr) run_floats<T>(load_run(z + t * a.z_stride + at[c], valid[c]), f);
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const bool in = k < valid[c];
        xh[c][k] = in ? __builtin_fmaf(xh[c][k], scale, -m) * r : 0.0f;
        const float u = __builtin_fmaf(xh[c][k], w[c][k], bias[c][k]);
        float slope, dn;
        if (z != nullptr) {
          dn = d[c][k] * act_of(a.act, f[k], slope);
          f[k] = d[c][k] * u * slope;
        } else {
          act_of(a.act, u, slope);
          dn = d[c][k] * slope;
        }
        if (!in) dn = 0.0f;
        dw[c][k] = __builtin_fmaf(dn, xh[c][k], dw[c][k]);
        db[c][k] += dn;
        d[c][k] = dn * w[c][k];
        s1 += d[c][k];
        s2 = __builtin_fmaf(d[c][k], xh[c][k], s2);
      }
      if (z != nullptr) store_run<T>(dz + t * a.dim + at[c], valid[c], f);
    }
    const float c1 = group_sum<LR>(s1, s_sum[0]) * rn, c2 = group_sum<LR>(s2, s_sum[1]) * rn;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      float f[kRun];
#pragma unroll
      for (int k = 0; k < kRun; ++k) f[k] = rstd * (d[c][k] - c1 - xh[c][k] * c2);
      store_run<T>(dx + t * a.dim + at[c], valid[c], f);
    }
  }
  if (a.part == nullptr) return;
  // the sums of the tokens side by side in the wave, then of the workgroup's waves
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t slice = group_index() / slabs;
  float* part = a.part + slice * 2 * a.dim;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int c = 0; c < K; ++c) {
      float f[kRun];
#pragma unroll
      for (int k = 0; k < kRun; ++k) f[k] = which == 0 ? dw[c][k] : db[c][k];
      if constexpr (LR <= 64) {
        if (p.per > 1) {
          const int lanes = a.groups * LR;
          int top = 1;
          while (2 * top < p.per) top *= 2;
          for (int off = top; off >= 1; off /= 2) {
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
              const float o = __shfl(f[k], (lane + off * lanes) & 63);
              if (p.sub < off && p.sub + off < p.per) f[k] += o;
            }
          }
        }
        __syncthreads();
        if (wave > 0) {
#pragma unroll
          for (int k = 0; k < kRun; ++k) s_acc[wave - 1][lane][k] = f[k];
        }
        __syncthreads();
        if (wave == 0) {
#pragma unroll
          for (int k = 0; k < kRun; ++k)
            for (int o = 0; o < kWaves - 1; ++o) f[k] += s_acc[o][lane][k];
        }
        if (wave != 0 || p.sub != 0) continue;
      }
      store_run<float>(part + which * (int64_t)a.dim + c0 + at[c], valid[c], f);
    }
  }
}

namespace {

// Lanes of a group and runs of a lane.
struct GroupPlan {
  int LR, K, slabs;
  int64_t slices;  // workgroups that go over the tokens of a slab
};

GroupPlan group_plan(int64_t tokens, int dim, int groups, bool bwd) {
  const int width = dim / groups;
  GroupPlan pl{1, 1, 1, 1};
  while (pl.LR < 64 && pl.LR * kRun < width) pl.LR *= 2;
  while (pl.K < 2 && pl.LR * pl.K * kRun < width) pl.K *= 2;
  if (pl.LR * pl.K * kRun < width) {
    pl.LR = 256;
    pl.K = width <= 256 * kRun ? 1 : width <= 256 * 2 * kRun ? 2 : 4;
  }
  const int team = pl.LR > 64 ? pl.LR : 64, teams = kBlockSpan / team;
  const int64_t lanes = (int64_t)groups * pl.LR;
  const int64_t per = lanes < team ? team / lanes : 1;
  pl.slabs = (int)((lanes + team - 1) / team);
  const int64_t rounds = (tokens + teams * per - 1) / (teams * per);  // workgroups that have a token
  const auto over = [&](int64_t n) { return (n + pl.slabs - 1) / pl.slabs; };
  pl.slices = over(kFwdGroups);
  if (bwd) pl.slices = std::min(over(kBwdGroups), std::max(over(kBwdLeast), tokens / kPartTokens));
  if (pl.slices > rounds) pl.slices = rounds;
  return pl;
}

template <typename T, int K, int LR>
hipError_t run(const GroupNormLaunch& a, const GroupPlan& pl, bool bwd, hipStream_t stream) {
  const dim3 grid = grid_of(pl.slabs * pl.slices, kBlockSpan);
  if (bwd) group_norm_bwd_kernel<T, K, LR><<<grid, kBlockSpan, 0, stream>>>(a, pl.slabs, pl.slices);
  else group_norm_fwd_kernel<T, K, LR><<<grid, kBlockSpan, 0, stream>>>(a, pl.slabs, pl.slices);
  return hipGetLastError();
}

template <typename T>
hipError_t run_plan(const GroupNormLaunch& a, const GroupPlan& pl, bool bwd, hipStream_t stream) {
  switch (pl.LR) {
    case 1: return run<T, 1, 1>(a, pl, bwd, stream);
    case 2: return run<T, 1, 2>(a, pl, bwd, stream);
    case 4: return run<T, 1, 4>(a, pl, bwd, stream);
    case 8: return run<T, 1, 8>(a, pl, bwd, stream);
    case 16: return run<T, 1, 16>(a, pl, bwd, stream);
    case 32: return run<T, 1, 32>(a, pl, bwd, stream);
    case 64:
      if (pl.K == 1) return run<T, 1, 64>(a, pl, bwd, stream);
      return run<T, 2, 64>(a, pl, bwd, stream);
  }
  if (pl.K == 1) return run<T, 1, 256>(a, pl, bwd, stream);
  return pl.K == 2 ? run<T, 2, 256>(a, pl, bwd, stream) : run<T, 4, 256>(a, pl, bwd, stream);
}

hipError_t launch(const GroupNormLaunch& a, bool bwd, hipStream_t stream) {
  const GroupPlan pl = group_plan(a.tokens, a.dim, a.groups, bwd);
  return a.dtype == Dtype::BF16 ? run_plan<uint16_t>(a, pl, bwd, stream) : run_plan<float>(a, pl, bwd, stream);
}

}  // namespace

int64_t group_norm_bwd_parts(int64_t tokens, int dim, int groups) { return group_plan(tokens, dim, groups, true).slices; }

hipError_t launch_group_norm_fwd(const GroupNormLaunch& a, hipStream_t stream) { return launch(a, false, stream); }

hipError_t launch_group_norm_bwd(const GroupNormLaunch& a, hipStream_t stream) {
  const hipError_t e = launch(a, true, stream);
  if (e != hipSuccess || a.part == nullptr) return e;
  return launch_norm_sum(a.part, a.dweight, a.dbias, (int)group_norm_bwd_parts(a.tokens, a.dim, a.groups), a.dim, stream);
}

}  // namespace ssm
