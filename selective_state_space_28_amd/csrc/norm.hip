// norm.hip -- layer norm over the channels of (batch, dim, seqlen), forward and
// backward, for gfx950 (include/ssm_norm.h states it).
//
// Both directions are bound by HBM: a few operations an element against 4 to 8
// bytes of bf16.  Two layouts:
//
//  * seqlen = 1, tokens with their channels together ("rows"): a row is held in
//    the registers of one workgroup slice of W waves (each lane kRun elements,
//    K times), so it is read once; the sums go over the lanes by DPP and over the
//    waves through LDS.
//  * seqlen > 1, the scans' layout ("columns"): a workgroup takes kTile
//    consecutive steps of a batch row and every channel; four lanes hold the
//    kTile steps of a channel, so an access of a wave is 16 pieces of 64 bytes
//    (bf16), and the sums over the channels go over 16 lanes and the waves.
//
// The mean is taken first and the variance about it, both in float32, as
// quotients by dim (a token of equal values has exactly that mean).
//
// dweight and dbias are sums over the tokens: each workgroup leaves its part
// (part[p][0] of dweight, part[p][1] of dbias) and norm_sum_kernel adds the
// parts in a fixed order.
#include "runs.hpp"
#include "ssm_kernels.hpp"

namespace ssm {

namespace {

constexpr int kMaxRowWaves = 16;  // waves of a row, at most one workgroup
constexpr int kTile = 32;         // steps of a column tile
constexpr int kTileLanes = kTile / kRun;
constexpr int kTileRows = 64 / kTileLanes;  // channels of one access of a wave
constexpr int kTileWaves = 16;
constexpr int kRowSpan = 64 * kRun;  // elements of one access of a wave

// Sum over the W waves of a row of a workgroup whose rows are `slot`s; every
// wave returns the total.  `s` is this sum's own LDS.
__device__ __forceinline__ float row_sum(float v, float (*s)[kMaxRowWaves], int slot, int wave, int W) {
  v = wave_sum(v);
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) s[slot][wave] = v;
  __syncthreads();
  float t = 0.0f;
  for (int k = 0; k < W; ++k) t += s[slot][k];
  return t;
}

// Channels of lane `l` of a row in its c-th access: first element.
__device__ __forceinline__ int row_at(int c, int l, int W) { return (c * W * 64 + l) * kRun; }

__device__ __forceinline__ void load_f32_run(const float* p, int valid, float (&f)[kRun]) {
  run_floats<float>(load_run<float>(p, valid), f);
}

}  // namespace

// Rows, forward.  Workgroup: 64 W threads a row, blockDim.x / (64 W) rows.
template <typename T, int K>
__global__ __launch_bounds__(1024) void norm_rows_fwd_kernel(
    const T* __restrict__ x, const T* __restrict__ residual, const float* __restrict__ weight,
    const float* __restrict__ bias, float eps, T* __restrict__ y, T* __restrict__ sum_out,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int rows, int dim, int W) {
  __shared__ float s_mean[4][kMaxRowWaves], s_var[4][kMaxRowWaves];
  const int span = W * 64;
  const int slot = __builtin_amdgcn_readfirstlane(threadIdx.x / span);
  const int l = threadIdx.x - slot * span;
  const int wave = l >> 6;
  const int row = blockIdx.x * (blockDim.x / span) + slot;
  const bool live = row < rows;  // idle rows run along to the barriers
  const int64_t base = (int64_t)(live ? row : 0) * dim;

  float v[K][kRun];
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int at = row_at(c, l, W);
    const int valid = live ? dim - at : 0;
    run_floats<T>(load_run(x + base + at, valid), v[c]);
    if (residual != nullptr) {
      float f[kRun];
      run_floats<T>(load_run(residual + base + at, valid), f);
#pragma unroll
      for (int k = 0; k < kRun; ++k) v[c][k] += f[k];
      store_run<T>(sum_out + base + at, valid, v[c]);
      // the norm is of the stream as stored
      if constexpr (sizeof(T) == 2) {
        RunWords<T> w;
        pack_floats<T, kRun>(v[c], w.w);
        run_floats<T>(w, v[c]);
      }
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k) sum += v[c][k];  // past the end: zeros
  }
  const float n = (float)dim;
  const float mean = row_sum(sum, s_mean, slot, wave, W) / n;
  float sq = 0.0f;
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int valid = dim - row_at(c, l, W);
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      v[c][k] -= mean;
      sq += k < valid ? v[c][k] * v[c][k] : 0.0f;
    }
  }
  const float rstd = 1.0f / __builtin_sqrtf(row_sum(sq, s_var, slot, wave, W) / n + eps);
  if (live && l == 0) {
    if (mean_out != nullptr) mean_out[row] = mean;
    if (rstd_out != nullptr) rstd_out[row] = rstd;
  }
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int at = row_at(c, l, W);
    const int valid = live ? dim - at : 0;
    float fw[kRun], fb[kRun];
    load_f32_run(weight + at, valid, fw);
    if (bias != nullptr) load_f32_run(bias + at, valid, fb);
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      v[c][k] = __builtin_fmaf(v[c][k] * rstd, fw[k], bias != nullptr ? fb[k] : 0.0f);
    store_run<T>(y + base + at, valid, v[c]);
  }
}

// Rows, backward: dx, and this slice's part of dweight and dbias.  A slice
// takes the rows slice, slice + slices, ...
template <typename T, int K>
__global__ __launch_bounds__(1024) void norm_rows_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* __restrict__ dy, const T* __restrict__ dsum, T* __restrict__ dx,
    float* __restrict__ part, int rows, int dim, int W, int slices) {
  __shared__ float s_a[2][4][kMaxRowWaves], s_b[2][4][kMaxRowWaves];
  const int span = W * 64;
  const int slot = __builtin_amdgcn_readfirstlane(threadIdx.x / span);
  const int l = threadIdx.x - slot * span;
  const int wave = l >> 6;
  const int slice = blockIdx.x * (blockDim.x / span) + slot;
  const int steps = (rows + slices - 1) / slices;  // the same for all, for the barriers

  float fw[K][kRun], aw[K][kRun], ab[K][kRun];
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int at = row_at(c, l, W);
    load_f32_run(weight + at, dim - at, fw[c]);
#pragma unroll
    for (int k = 0; k < kRun; ++k) aw[c][k] = ab[c][k] = 0.0f;
  }
  const float n = (float)dim;
  for (int it = 0; it < steps; ++it) {
    const int64_t row = slice + (int64_t)it * slices;
    const bool live = slice < slices && row < rows;
    const int64_t base = (live ? row : 0) * dim;
    const float mu = live ? mean[row] : 0.0f, rs = live ? rstd[row] : 0.0f;
    float xh[K][kRun], g[K][kRun];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      const int at = row_at(c, l, W);
      const int valid = live ? dim - at : 0;
      run_floats<T>(load_run(x + base + at, valid), xh[c]);
      run_floats<T>(load_run(dy + base + at, valid), g[c]);
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        xh[c][k] = (xh[c][k] - mu) * rs;
        aw[c][k] = __builtin_fmaf(g[c][k], xh[c][k], aw[c][k]);  // past the end: dy is 0
        ab[c][k] += g[c][k];
        g[c][k] *= fw[c][k];
        c1 += g[c][k];
        c2 = __builtin_fmaf(g[c][k], xh[c][k], c2);
      }
    }
    c1 = row_sum(c1, s_a[it & 1], slot, wave, W) / n;
    c2 = row_sum(c2, s_b[it & 1], slot, wave, W) / n;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      const int at = row_at(c, l, W);
      const int valid = live ? dim - at : 0;
#pragma unroll
      for (int k = 0; k < kRun; ++k) g[c][k] = rs * (g[c][k] - c1 - xh[c][k] * c2);
      if (dsum != nullptr) {
        float f[kRun];
        run_floats<T>(load_run(dsum + base + at, valid), f);
#pragma unroll
        for (int k = 0; k < kRun; ++k) g[c][k] += f[k];
      }
      store_run<T>(dx + base + at, valid, g[c]);
    }
  }
  if (slice >= slices) return;
  float* const pw = part + (int64_t)slice * 2 * dim;
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int at = row_at(c, l, W);
    store_run<float>(pw + at, dim - at, aw[c]);
    store_run<float>(pw + dim + at, dim - at, ab[c]);
  }
}

namespace {

// ---- columns ---------------------------------------------------------------------
// A thread's place in a tile: steps t .. t + kRun - 1 of the channels d0, d0 +
// stride, ...
struct TilePlace {
  int b, t, valid, d0, stride, wave, lane;
  int64_t base;  // of channel 0 at step t
};

__device__ __forceinline__ TilePlace tile_place(int dim, int seqlen, int tiles) {
  TilePlace p;
  p.lane = threadIdx.x & 63;
  p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  p.b = blockIdx.x / tiles;
  p.t = (blockIdx.x - p.b * tiles) * kTile + (p.lane % kTileLanes) * kRun;
  p.valid = seqlen - p.t;
  p.d0 = p.wave * kTileRows + p.lane / kTileLanes;
  p.stride = (blockDim.x >> 6) * kTileRows;
  p.base = (int64_t)p.b * dim * seqlen + p.t;
  return p;
}

// Sums over the channels of NV values of each step: over the lanes that hold
// the same steps, then over the waves through LDS (its own per call).  The
// order is fixed.
template <int NV>
__device__ __forceinline__ void tile_sums(float (&v)[NV][kRun], float (*s)[NV][kTile], const TilePlace& p) {
#pragma unroll
  for (int q = 0; q < NV; ++q) {
#pragma unroll
    for (int k = 0; k < kRun; ++k)
#pragma unroll
      for (int off = kTileLanes; off < 64; off <<= 1) v[q][k] += __shfl_xor(v[q][k], off);
    if (p.lane < kTileLanes) {
#pragma unroll
      for (int k = 0; k < kRun; ++k) s[p.wave][q][p.lane * kRun + k] = v[q][k];
    }
  }
  __syncthreads();
  const int waves = blockDim.x >> 6;
#pragma unroll
  for (int q = 0; q < NV; ++q)
#pragma unroll
    for (int k = 0; k < kRun; ++k) v[q][k] = 0.0f;
  for (int w = 0; w < waves; ++w)
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int k = 0; k < kRun; ++k) v[q][k] += s[w][q][(p.lane % kTileLanes) * kRun + k];
}

}  // namespace

// Columns, forward.
template <typename T>
__global__ __launch_bounds__(64 * kTileWaves) void norm_cols_fwd_kernel(
    const T* __restrict__ x, const T* __restrict__ residual, const float* __restrict__ weight,
    const float* __restrict__ bias, float eps, T* __restrict__ y, T* sum_out,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int dim, int seqlen, int tiles) {
  __shared__ float s_mean[kTileWaves][1][kTile], s_var[kTileWaves][1][kTile];
  const TilePlace p = tile_place(dim, seqlen, tiles);
  const T* src = residual != nullptr ? sum_out : x;
  float mean[1][kRun], var[1][kRun];
#pragma unroll
  for (int k = 0; k < kRun; ++k) mean[0][k] = var[0][k] = 0.0f;
  for (int d = p.d0; d < dim; d += p.stride) {
    const int64_t at = p.base + (int64_t)d * seqlen;
    float f[kRun];
    run_floats<T>(load_run(x + at, p.valid), f);
    if (residual != nullptr) {
      float g[kRun];
      run_floats<T>(load_run(residual + at, p.valid), g);
#pragma unroll
      for (int k = 0; k < kRun; ++k) f[k] += g[k];
      store_run<T>(sum_out + at, p.valid, f);
      if constexpr (sizeof(T) == 2) {
        RunWords<T> w;
        pack_floats<T, kRun>(f, w.w);
        run_floats<T>(w, f);
      }
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k) mean[0][k] += f[k];
  }
  tile_sums<1>(mean, s_mean, p);
  const float n = (float)dim;
#pragma unroll
  for (int k = 0; k < kRun; ++k) mean[0][k] /= n;
  for (int d = p.d0; d < dim; d += p.stride) {
    float f[kRun];
    run_floats<T>(load_run(src + p.base + (int64_t)d * seqlen, p.valid), f);
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const float c = f[k] - mean[0][k];
      var[0][k] = __builtin_fmaf(c, c, var[0][k]);
    }
  }
  tile_sums<1>(var, s_var, p);
#pragma unroll
  for (int k = 0; k < kRun; ++k) var[0][k] = 1.0f / __builtin_sqrtf(var[0][k] / n + eps);
  if (p.wave == 0 && p.lane < kTileLanes) {
    const int64_t at = (int64_t)p.b * seqlen + p.t;
    if (mean_out != nullptr) store_run<float>(mean_out + at, p.valid, mean[0]);
    if (rstd_out != nullptr) store_run<float>(rstd_out + at, p.valid, var[0]);
  }
  for (int d = p.d0; d < dim; d += p.stride) {
    const int64_t at = p.base + (int64_t)d * seqlen;
    const float w = weight[d], b = bias != nullptr ? bias[d] : 0.0f;
    float f[kRun];
    run_floats<T>(load_run(src + at, p.valid), f);
#pragma unroll
    for (int k = 0; k < kRun; ++k) f[k] = __builtin_fmaf((f[k] - mean[0][k]) * var[0][k], w, b);
    store_run<T>(y + at, p.valid, f);
  }
}

// Columns, backward: dx, and this tile's part of dweight and dbias.
template <typename T>
__global__ __launch_bounds__(64 * kTileWaves) void norm_cols_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const T* __restrict__ dy, const T* __restrict__ dsum,
    T* __restrict__ dx, float* __restrict__ part, int dim, int seqlen, int tiles) {
  __shared__ float s_c[kTileWaves][2][kTile];
  const TilePlace p = tile_place(dim, seqlen, tiles);
  float mu[kRun], rs[kRun], c[2][kRun];
  load_f32_run(mean_in + (int64_t)p.b * seqlen + p.t, p.valid, mu);
  load_f32_run(rstd_in + (int64_t)p.b * seqlen + p.t, p.valid, rs);
#pragma unroll
  for (int k = 0; k < kRun; ++k) c[0][k] = c[1][k] = 0.0f;
  float* const pw = part + (int64_t)blockIdx.x * 2 * dim;
  // whole waves stay in the loop for the shuffles
  for (int dw = p.wave * kTileRows; dw < dim; dw += p.stride) {
    const int d = dw + p.lane / kTileLanes;
    const bool live = d < dim;
    const int64_t at = p.base + (int64_t)(live ? d : 0) * seqlen;
    const int valid = live ? p.valid : 0;
    const float w = live ? weight[d] : 0.0f;
    float f[kRun], g[kRun], sw = 0.0f, sb = 0.0f;
    run_floats<T>(load_run(x + at, valid), f);
    run_floats<T>(load_run(dy + at, valid), g);
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const float xh = (f[k] - mu[k]) * rs[k];
      sw = __builtin_fmaf(g[k], xh, sw);  // past the end: dy is 0
      sb += g[k];
      c[0][k] = __builtin_fmaf(g[k], w, c[0][k]);
      c[1][k] = __builtin_fmaf(g[k] * w, xh, c[1][k]);
    }
#pragma unroll
    for (int off = 1; off < kTileLanes; off <<= 1) {
      sw += __shfl_xor(sw, off);
      sb += __shfl_xor(sb, off);
    }
    if (live && p.lane % kTileLanes == 0) {
      pw[d] = sw;
      pw[dim + d] = sb;
    }
  }
  tile_sums<2>(c, s_c, p);
  const float n = (float)dim;
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    c[0][k] /= n;
    c[1][k] /= n;
  }
  for (int d = p.d0; d < dim; d += p.stride) {
    const int64_t at = p.base + (int64_t)d * seqlen;
    const float w = weight[d];
    float f[kRun], g[kRun];
    run_floats<T>(load_run(x + at, p.valid), f);
    run_floats<T>(load_run(dy + at, p.valid), g);
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const float xh = (f[k] - mu[k]) * rs[k];
      g[k] = rs[k] * (g[k] * w - c[0][k] - xh * c[1][k]);
    }
    if (dsum != nullptr) {
      run_floats<T>(load_run(dsum + at, p.valid), f);
#pragma unroll
      for (int k = 0; k < kRun; ++k) g[k] += f[k];
    }
    store_run<T>(dx + at, p.valid, g);
  }
}

// dweight[d] = sum_p part[p][0][d], dbias[d] = sum_p part[p][1][d].  A
// workgroup takes 32 of the 2 dim sums, 32 threads each.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* __restrict__ part, float* __restrict__ dweight,
                                                        float* __restrict__ dbias, int parts, int dim) {
  __shared__ float s[32][33];
  const int64_t at = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
  const int j = threadIdx.x >> 5;
  float v = 0.0f;
  if (at < 2 * (int64_t)dim)
    for (int p = j; p < parts; p += 32) v += part[(int64_t)p * 2 * dim + at];
  s[j][threadIdx.x & 31] = v;
  __syncthreads();
  if (j == 0 && at < 2 * (int64_t)dim) {
    float t = 0.0f;
    for (int k = 0; k < 32; ++k) t += s[k][threadIdx.x];
    if (at < dim) dweight[at] = t;
    else if (dbias != nullptr) dbias[at - dim] = t;
  }
}

namespace {

// Rows: waves of a row and accesses of a lane (1, 2 or 4; 0: a row too long
// for the registers of a workgroup), rows of a workgroup.
struct RowPlan {
  int W, K, rows;
};

RowPlan row_plan(int dim) {
  const int spans = (dim + kRowSpan - 1) / kRowSpan;
  int K = 1;
  while (K < 4 && spans > kMaxRowWaves * K) K *= 2;
  if (spans > kMaxRowWaves * K) return RowPlan{0, 0, 0};
  const int W = (spans + K - 1) / K;
  return RowPlan{W, K, W >= 4 ? 1 : 4 / W};
}

// Slices of the rows' backward: enough workgroups to fill the chip, and 16
// rows to a slice so that the parts stay small beside the rows.
int row_slices(int rows) {
  const int most = 1024;
  const int s = (rows + 15) / 16;
  return s < most ? s : most;
}

int tiles_of(int64_t seqlen) { return (int)((seqlen + kTile - 1) / kTile); }

unsigned tile_threads(int dim) {
  const int waves = (dim + kTileRows - 1) / kTileRows;
  return 64u * (unsigned)(waves < kTileWaves ? waves : kTileWaves);
}

template <typename T, int K>
hipError_t rows_fwd(const NormLaunch& a, const RowPlan& pl, hipStream_t stream) {
  const unsigned grid = (unsigned)((a.batch + pl.rows - 1) / pl.rows);
  norm_rows_fwd_kernel<T, K><<<grid, 64 * pl.W * pl.rows, 0, stream>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.residual), a.weight, a.bias, a.eps,
      static_cast<T*>(a.y), static_cast<T*>(a.sum_out), a.mean, a.rstd, a.batch, a.dim, pl.W);
  return hipGetLastError();
}

template <typename T, int K>
hipError_t rows_bwd(const NormLaunch& a, const RowPlan& pl, hipStream_t stream) {
  const int slices = row_slices(a.batch);
  const unsigned grid = (unsigned)((slices + pl.rows - 1) / pl.rows);
  norm_rows_bwd_kernel<T, K><<<grid, 64 * pl.W * pl.rows, 0, stream>>>(
      static_cast<const T*>(a.x), a.weight, a.mean, a.rstd, static_cast<const T*>(a.dy),
      static_cast<const T*>(a.dsum), static_cast<T*>(a.dx), a.part, a.batch, a.dim, pl.W, slices);
  return hipGetLastError();
}

template <typename T>
hipError_t fwd_typed(const NormLaunch& a, hipStream_t stream) {
  const RowPlan pl = row_plan(a.dim);
  if (a.seqlen == 1 && pl.K > 0) {
    switch (pl.K) {
      case 1: return rows_fwd<T, 1>(a, pl, stream);
      case 2: return rows_fwd<T, 2>(a, pl, stream);
      default: return rows_fwd<T, 4>(a, pl, stream);
    }
  }
  const int tiles = tiles_of(a.seqlen);
  norm_cols_fwd_kernel<T><<<(unsigned)(a.batch * tiles), tile_threads(a.dim), 0, stream>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.residual), a.weight, a.bias, a.eps,
      static_cast<T*>(a.y), static_cast<T*>(a.sum_out), a.mean, a.rstd, a.dim, (int)a.seqlen, tiles);
  return hipGetLastError();
}

template <typename T>
hipError_t bwd_typed(const NormLaunch& a, hipStream_t stream) {
  const RowPlan pl = row_plan(a.dim);
  hipError_t e;
  if (a.seqlen == 1 && pl.K > 0) {
    e = pl.K == 1 ? rows_bwd<T, 1>(a, pl, stream)
                  : pl.K == 2 ? rows_bwd<T, 2>(a, pl, stream) : rows_bwd<T, 4>(a, pl, stream);
  } else {
    const int tiles = tiles_of(a.seqlen);
    norm_cols_bwd_kernel<T><<<(unsigned)(a.batch * tiles), tile_threads(a.dim), 0, stream>>>(
        static_cast<const T*>(a.x), a.weight, a.mean, a.rstd, static_cast<const T*>(a.dy),
        static_cast<const T*>(a.dsum), static_cast<T*>(a.dx), a.part, a.dim, (int)a.seqlen, tiles);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  const int parts = norm_bwd_parts(a.batch, a.dim, a.seqlen);
  norm_sum_kernel<<<(unsigned)((2 * (int64_t)a.dim + 31) / 32), 1024, 0, stream>>>(a.part, a.dweight, a.dbias,
                                                                                   parts, a.dim);
  return hipGetLastError();
}

}  // namespace

int norm_bwd_parts(int batch, int dim, int64_t seqlen) {
  if (seqlen == 1 && row_plan(dim).K > 0) return row_slices(batch);
  return batch * tiles_of(seqlen);
}

hipError_t launch_norm_fwd(const NormLaunch& a, hipStream_t stream) {
  return a.dtype == Dtype::BF16 ? fwd_typed<uint16_t>(a, stream) : fwd_typed<float>(a, stream);
}

hipError_t launch_norm_bwd(const NormLaunch& a, hipStream_t stream) {
  return a.dtype == Dtype::BF16 ? bwd_typed<uint16_t>(a, stream) : bwd_typed<float>(a, stream);
}

}  // namespace ssm
