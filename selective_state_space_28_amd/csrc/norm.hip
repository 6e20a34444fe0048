// norm.hip -- layer norm over the channels of (batch, dim, seqlen), forward and
// backward, for gfx950 (include/ssm_norm.h states it).
//
// Both directions are bound by HBM: a few operations an element against 4 to 8
// bytes of bf16.  Two layouts:
//
//  * seqlen = 1, tokens with their channels together ("rows"): a row is held in
//    the registers of 8 lanes to 16 waves (each lane kRun elements, K times), so
//    it is read once; the sums go over the lanes by DPP and over the waves
//    through LDS.
//  * seqlen > 1, the scans' layout ("columns"): a workgroup takes a tile of
//    consecutive steps of a batch row and every channel; TL lanes of 16 bytes side
//    by side hold a channel's steps of the tile, so an access of a wave is 64/TL
//    pieces of 16 TL bytes.  It goes over the tile twice, once for the sums over
//    the channels and once for the results.
//
// The mean is taken first and the variance about it.  A token of equal values has
// exactly that mean: a column's is a running one, and where values are summed and
// divided by dim their sum is exact, in float32 of up to 2^16 values of bf16 (8
// bits), in float64 otherwise (rows of float32, columns of a few steps).
//
// dweight and dbias are sums over the tokens: each workgroup leaves its part
// (part[p][0] of dweight, part[p][1] of dbias) and norm_sum_kernel adds the
// parts in a fixed order.
#include "runs.hpp"
#include "ssm_kernels.hpp"

namespace ssm {

namespace {

constexpr int kMaxRowWaves = 16;  // waves of a row, at most one workgroup
constexpr int kTileWaves = 8;    // most waves of a column tile
constexpr int kRowSpan = 64 * kRun;  // elements of one access of a wave

// Sum over a row, in every lane of it: over its LR lanes, and over the W waves
// of a row longer than a wave (LR = 64), the `slot`-th of its workgroup.  `s` is
// this sum's own LDS.  The order is fixed.  V: float or double.
template <int LR = 64, typename V>
__device__ __forceinline__ V row_sum(V v, V (*s)[kMaxRowWaves], int slot, int wave, int W) {
  if constexpr (LR < 64) {
    v += dpp_moved<0xb1, 0xf>(v);   // quad_perm: the pair's other
    v += dpp_moved<0x4e, 0xf>(v);   // quad_perm: the other pair
    v += dpp_moved<0x141, 0xf>(v);  // row_half_mirror: the other 4 of 8
    if constexpr (LR >= 16) v += dpp_moved<0x140, 0xf>(v);  // row_mirror: the other 8 of 16
    if constexpr (LR >= 32) v += __shfl_xor(v, 16);
    return v;
  }
  v = wave_sum(v);
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) s[slot][wave] = v;
  __syncthreads();
  V t = 0;
  for (int k = 0; k < W; ++k) t += s[slot][k];
  return t;
}

// What a row's values of T are summed in: exact for equal values, and inside the
// type's range (tokens masked by the lowest value): a float32 holds the sum of 16-bit
// values 2^-16 times its size, which costs neither bits nor an instruction.
template <typename T>
using RowSum = typename std::conditional<sizeof(T) == 4, double, float>::type;
constexpr float kSumScale = 1.0f / 65536;

__device__ __forceinline__ void load_f32_run(const float* p, int valid, float (&f)[kRun]) {
  run_floats<float>(load_run<float>(p, valid), f);
}

}  // namespace

// A thread's place among the rows of a workgroup: slot of the row, lane in it.
template <int LR>
struct RowPlace {
  int slot, lane, wave, slots, span;  // span: lanes of a row
};

template <int LR>
__device__ __forceinline__ RowPlace<LR> row_place(int W) {
  RowPlace<LR> p;
  p.span = LR < 64 ? LR : W * 64;
  p.slot = (int)threadIdx.x / p.span;
  if constexpr (LR == 64) p.slot = __builtin_amdgcn_readfirstlane(p.slot);
  p.lane = threadIdx.x - p.slot * p.span;
  p.wave = p.lane >> 6;
  p.slots = (int)blockDim.x / p.span;
  return p;
}

// Rows, forward.  A row takes LR lanes (up to 8 LR channels) or 64 W, each lane
// kRun channels K times; the workgroup's other threads other rows; rn = 1 / dim.
// 16-bit results go past the caches (32768 rows of 2560 bf16: 88 us, through them
// 107; float32's two stores of a run fill a line only together: 16384 rows of 1000
// 48 us, through the caches 43).
template <typename T, int K, int LR>
__global__ __launch_bounds__(1024) void norm_rows_fwd_kernel(
    const T* __restrict__ x, const T* __restrict__ residual, const float* __restrict__ weight,
    const float* __restrict__ bias, float eps, T* __restrict__ y, T* __restrict__ sum_out,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int rows, int dim, double rn, int W) {
  __shared__ RowSum<T> s_mean[4][kMaxRowWaves];
  __shared__ float s_var[4][kMaxRowWaves];
  const RowPlace<LR> p = row_place<LR>(W);
  const int64_t row = group_index() * p.slots + p.slot;
  const bool live = row < rows;  // idle rows run along to the barriers
  const int64_t base = (live ? row : 0) * dim;

  float v[K][kRun];
  RowSum<T> sum = 0;
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int at = (c * p.span + p.lane) * kRun;
    const int valid = live ? dim - at : 0;
    run_floats<T>(load_run(x + base + at, valid), v[c]);
    if (residual != nullptr) {
      float f[kRun];
      run_floats<T>(load_run(residual + base + at, valid), f);
#pragma unroll
      for (int k = 0; k < kRun; ++k) v[c][k] += f[k];
      store_run<T, sizeof(T) == 2>(sum_out + base + at, valid, v[c]);
      // the norm is of the stream as stored
      if constexpr (sizeof(T) == 2) {
        RunWords<T> w;
        pack_floats<T, kRun>(v[c], w.w);
        run_floats<T>(w, v[c]);
      }
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k)  // past the end: zeros
      sum = sizeof(T) == 4 ? sum + v[c][k] : __builtin_fmaf(v[c][k], kSumScale, sum);
  }
  const float n = (float)dim;
  sum = row_sum<LR>(sum, s_mean, p.slot, p.wave, W);
  // (a division in float64 is some 15 instructions; the product's two roundings
  // to 53 bits do not reach the 24 of equal values' mean)
  const float mean = sizeof(T) == 4 ? (float)(sum * rn) : (float)sum / n * (1.0f / kSumScale);
  float sq = 0.0f;
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int valid = dim - (c * p.span + p.lane) * kRun;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      v[c][k] -= mean;
      sq += k < valid ? v[c][k] * v[c][k] : 0.0f;
    }
  }
  const float rstd = 1.0f / __builtin_sqrtf(row_sum<LR>(sq, s_var, p.slot, p.wave, W) / n + eps);
  if (live && p.lane == 0) {
    if (mean_out != nullptr) mean_out[row] = mean;
    if (rstd_out != nullptr) rstd_out[row] = rstd;
  }
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int at = (c * p.span + p.lane) * kRun;
    const int valid = live ? dim - at : 0;
    float fw[kRun], fb[kRun];
    load_f32_run(weight + at, valid, fw);
    if (bias != nullptr) load_f32_run(bias + at, valid, fb);
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      v[c][k] = __builtin_fmaf(v[c][k] * rstd, fw[k], bias != nullptr ? fb[k] : 0.0f);
    store_run<T, sizeof(T) == 2>(y + base + at, valid, v[c]);
  }
}

// Rows, backward: dx, and this workgroup's part of dweight and dbias.  A
// workgroup's rows are its slots', then those gridDim.x workgroups on; its
// slots' sums are added in order in LDS (s_acc, 2 dim floats a slot; one slot: none).
template <typename T, int K, int LR>
__global__ __launch_bounds__(1024) void norm_rows_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* __restrict__ dy, const T* __restrict__ dsum, T* __restrict__ dx,
    float* __restrict__ part, int rows, int dim, int W) {
  __shared__ float s_a[2][kMaxRowWaves][kMaxRowWaves], s_b[2][kMaxRowWaves][kMaxRowWaves];
  extern __shared__ float s_acc[];
  const RowPlace<LR> p = row_place<LR>(W);
  const int all = (int)gridDim.x * p.slots;       // rows of one turn
  const int turns = (rows - 1) / all + 1;         // the same for all, for the barriers

  float fw[K][kRun], aw[K][kRun], ab[K][kRun];
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int at = (c * p.span + p.lane) * kRun;
    load_f32_run(weight + at, dim - at, fw[c]);
#pragma unroll
    for (int k = 0; k < kRun; ++k) aw[c][k] = ab[c][k] = 0.0f;
  }
  const float n = (float)dim;
  // a row's inputs, read a turn ahead
  RunWords<T> wx[K], wd[K];
  float mu_n = 0.0f, rs_n = 0.0f;
  auto fetch = [&](int it) {
    const int64_t row = (int64_t)it * all + (int64_t)blockIdx.x * p.slots + p.slot;
    const bool live = row < rows;
    mu_n = live ? mean[row] : 0.0f;
    rs_n = live ? rstd[row] : 0.0f;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      const int at = (c * p.span + p.lane) * kRun;
      const int64_t from = (live ? row : 0) * dim + at;
      wx[c] = load_run(x + from, live ? dim - at : 0);
      wd[c] = load_run(dy + from, live ? dim - at : 0);
    }
  };
  fetch(0);
  for (int it = 0; it < turns; ++it) {
    const int64_t row = (int64_t)it * all + (int64_t)blockIdx.x * p.slots + p.slot;
    const bool live = row < rows;
    const int64_t base = (live ? row : 0) * dim;
    const float mu = mu_n, rs = rs_n;
    float xh[K][kRun], g[K][kRun];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      run_floats<T>(wx[c], xh[c]);
      run_floats<T>(wd[c], g[c]);
      // Past the end dy is 0, but a zero less a far mean, times rstd, may be infinite:
      // x is the mean there.
      const int at = (c * p.span + p.lane) * kRun;
      if (dim - at < kRun) {
#pragma unroll
        for (int k = 0; k < kRun; ++k) xh[c][k] = at + k < dim ? xh[c][k] : mu;
      }
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
    if (it + 1 < turns) fetch(it + 1);
    c1 = row_sum<LR>(c1, s_a[it & 1], p.slot, p.wave, W) / n;
    c2 = row_sum<LR>(c2, s_b[it & 1], p.slot, p.wave, W) / n;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      const int at = (c * p.span + p.lane) * kRun;
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
  float* const pw = part + (int64_t)blockIdx.x * 2 * dim;
  if (p.slots == 1) {
#pragma unroll
    for (int c = 0; c < K; ++c) {
      const int at = (c * p.span + p.lane) * kRun;
      store_run<float>(pw + at, dim - at, aw[c]);
      store_run<float>(pw + dim + at, dim - at, ab[c]);
    }
    return;
  }
  float* const own = s_acc + (int64_t)p.slot * 2 * dim;
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int at = (c * p.span + p.lane) * kRun;
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      if (at + k < dim) {
        own[at + k] = aw[c][k];
        own[dim + at + k] = ab[c][k];
      }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < 2 * dim; k += blockDim.x) {
    float t = 0.0f;
    for (int slot = 0; slot < p.slots; ++slot) t += s_acc[slot * 2 * dim + k];
    pw[k] = t;
  }
}

namespace {

// ---- columns ---------------------------------------------------------------------
// 16 bytes of consecutive elements.
template <typename T>
struct Piece {
  static constexpr int kN = 16 / (int)sizeof(T);
  uint32_t w[4];
  __device__ __forceinline__ void floats(float (&f)[kN]) const { words_to_floats<T, kN>(w, f); }
  __device__ __forceinline__ void set(const float (&f)[kN]) { pack_floats<T, kN>(f, w); }
  // The words as if written anew: what was derived from them (their elements
  // as floats, twice the registers) is formed again instead of kept from one
  // pass over the tile to the next.
  __device__ __forceinline__ void renew() { asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3])); }
};

// The same for a scalar that a loop does not change: what follows from it (an
// index for each access) is formed in each turn instead of held across them.
__device__ __forceinline__ int renewed(int v) {
  asm volatile("" : "+s"(v));
  return v;
}

// Holds v formed here: with the words renewed after it, what was unpacked for it is dead by then.
__device__ __forceinline__ void settle(float& v) { asm volatile("" : "+v"(v)); }

// Where the row has a whole piece (seqlen >= kN), a piece that would pass the
// row's end is moved back to end with it: every access is whole, and its first
// `dup` steps are those of the lanes before, computed again here and neither
// stored nor counted.  An address is a part that the wave shares (the batch row
// and the access' first channel, in scalar registers) and the lane's byte offset
// `at`, the same for every access.
struct WholePlace {
  int dup;        // 0 .. kN
  bool ragged;    // the tile has pieces with dup > 0
  uint32_t at;    // byte offset of the lane's channel among the access' and of its step
  int64_t row, token;
};

template <typename T, int TL>
__device__ __forceinline__ WholePlace whole_place(int tile, int dim, int seqlen, int tiles, int lane) {
  constexpr int E = Piece<T>::kN;
  WholePlace p;
  const int b = tile / tiles;
  const int t0 = (tile - b * tiles) * TL * E;
  const int over = t0 + (lane % TL + 1) * E - seqlen;
  p.dup = over <= 0 ? 0 : over < E ? over : E;
  p.ragged = t0 + TL * E > seqlen;
  const int t = over <= 0 ? t0 + lane % TL * E : seqlen - E;
  p.at = (uint32_t)(lane / TL) * (uint32_t)seqlen * (uint32_t)sizeof(T) + (uint32_t)t * (uint32_t)sizeof(T);
  p.row = (int64_t)b * dim * seqlen;
  p.token = (int64_t)b * seqlen + t;
  return p;
}

template <typename T>
__device__ __forceinline__ const T* at_bytes(const T* p, uint32_t bytes) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + bytes);
}
template <typename T>
__device__ __forceinline__ T* at_bytes(T* p, uint32_t bytes) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(p) + bytes);
}

template <typename T>
__device__ __forceinline__ Piece<T> load_whole(const T* p) {
  const auto v = *reinterpret_cast<const typename RunWords<T>::vec4*>(p);
  Piece<T> r;
  r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  return r;
}

// An access' first channel: one that would pass the last channel is moved back
// to end with it (dim >= rows), and its channels before dw, which other accesses
// hold, are not live.  So every address is a scalar part plus the lane's offset.
__device__ __forceinline__ int inside(int dw, int rows, int dim) { return dw + rows <= dim ? dw : dim - rows; }

// Store what the piece does not share with the lanes before.  `once`: the
// access' pieces are whole lines and not read back, so they need not displace
// the inputs that are read again (batch 16, dim 5120, L 2048 bf16: 164 us
// against 201; with rows that straddle lines, which the L2 then joins, it costs
// more than it gives: batch 8, dim 1536, L 2047 float32, backward, 99 us against 88).
template <typename T>
__device__ __forceinline__ void store_whole(T* p, const WholePlace& h, const float (&f)[Piece<T>::kN], bool once) {
  if (!h.ragged) {
    Piece<T> r;
    r.set(f);
    const typename RunWords<T>::vec4 v = {r.w[0], r.w[1], r.w[2], r.w[3]};
    if (once) {
      asm volatile("; once");  // keeps the two stores from being merged into a plain one
      __builtin_nontemporal_store(v, reinterpret_cast<typename RunWords<T>::vec4*>(p));
      asm volatile("; once");
    } else {
      *reinterpret_cast<typename RunWords<T>::vec4*>(p) = v;
    }
  } else {
#pragma unroll
    for (int q = 0; q < Piece<T>::kN; ++q)
      if (q >= h.dup) Elem<T>::store(p + q, f[q]);
  }
}

// Workgroups go to the 8 XCDs in turn; tiles side by side share lines (128
// bytes, a tile's piece is 32 to 128, and rows of any length straddle them), so
// those that run together are given to one XCD's L2: the block's place in an
// order that keeps an XCD's blocks together.
__device__ __forceinline__ int xcd_order(int block, int blocks) {
  const int per = blocks / 8;
  return block < per * 8 ? (block % 8) * per + block / 8 : block;
}

// Mean and sum of squares about it of n values, per step, and their union with
// those of others (mb, sb of nb values): no difference of large squares.
template <int E>
struct Spread {
  float n, mean[E], sq[E];
  __device__ __forceinline__ void clear() {
    n = 0.0f;
#pragma unroll
    for (int k = 0; k < E; ++k) mean[k] = sq[k] = 0.0f;
  }
  // one more value per step; rn = 1 / (n + 1)
  __device__ __forceinline__ void add(const float (&f)[E], float rn) {
    n += 1.0f;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float d = f[k] - mean[k];
      mean[k] = __builtin_fmaf(d, rn, mean[k]);
      sq[k] = __builtin_fmaf(d, f[k] - mean[k], sq[k]);
    }
  }
  __device__ __forceinline__ void join(float nb, const float (&mb)[E], const float (&sb)[E]) {
    const float all = n + nb;
    const float share = all > 0.0f ? nb / all : 0.0f, both = n * share;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float d = mb[k] - mean[k];
      mean[k] = __builtin_fmaf(d, share, mean[k]);
      // Where a side has no values d is the other's mean, whose square may be
      // infinite: it has no part.
      const float apart = both > 0.0f ? d : 0.0f;
      sq[k] += __builtin_fmaf(apart * apart, both, sb[k]);
    }
    n = all;
  }
};

}  // namespace

namespace {

// Sums of n values over the lanes that hold the same steps: every TL-th lane.
// In a row of 16 lanes the rotations give each lane the others', across rows
// the exchange; the order is fixed.
template <int OFF>
__device__ __forceinline__ float from_lane(float v) {
  if constexpr (OFF < 16) return dpp_moved<0x120 + OFF, 0xf>(v);  // row_ror
  else return __shfl_xor(v, OFF);
}

template <int OFF, int E>
__device__ __forceinline__ void join_lanes(Spread<E>& a) {
  if constexpr (OFF < 64) {
    float m[E], q[E];
    const float n = from_lane<OFF>(a.n);
#pragma unroll
    for (int k = 0; k < E; ++k) {
      m[k] = from_lane<OFF>(a.mean[k]);
      q[k] = from_lane<OFF>(a.sq[k]);
    }
    a.join(n, m, q);
    join_lanes<2 * OFF, E>(a);
  }
}

template <int OFF, int N>
__device__ __forceinline__ void add_lanes(float (&v)[N]) {
  if constexpr (OFF < 64) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += from_lane<OFF>(v[k]);
    add_lanes<2 * OFF, N>(v);
  }
}

// A lane's piece kept in LDS, and read back.
template <typename T>
__device__ __forceinline__ void keep(uint4* s, const Piece<T>& v) {
  *s = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}
template <typename T>
__device__ __forceinline__ Piece<T> kept_piece(const uint4* s) {
  const uint4 v = *s;
  Piece<T> r;
  r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  return r;
}

// Floats of LDS that n parameters of the channels take, in whole pieces.
__host__ __device__ constexpr int param_floats(int n, int dim) { return (n * dim + 3) / 4 * 4; }

// The spread of each step of a tile over the workgroup's waves: what every lane's
// own spread (its channels) joins to.  mean and rstd of the lane's steps come
// back, and go to mean_out and rstd_out.  Two barriers.
template <typename T, int TL>
struct TileStats {
  static constexpr int E = Piece<T>::kN;
  float n[kTileWaves], part[kTileWaves][2][TL * E], stat[2][TL * E];
};

template <typename T, int TL>
__device__ __forceinline__ void tile_stats(Spread<Piece<T>::kN>& sp, TileStats<T, TL>& s, float eps, int tile, int dim,
                                           int seqlen, int tiles, float* mean_out, float* rstd_out,
                                           float (&mean)[Piece<T>::kN], float (&rstd)[Piece<T>::kN]) {
  constexpr int E = Piece<T>::kN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  join_lanes<TL, E>(sp);
  if (lane < TL) {
    s.n[wave] = sp.n;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      s.part[wave][0][lane * E + k] = sp.mean[k];
      s.part[wave][1][lane * E + k] = sp.sq[k];
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < TL * E; j += blockDim.x) {
    Spread<1> all;
    all.clear();
    for (int w = 0; w < waves; ++w) {
      const float m[1] = {s.part[w][0][j]}, q[1] = {s.part[w][1][j]};
      all.join(s.n[w], m, q);
    }
    const float rs = 1.0f / __builtin_sqrtf(all.sq[0] / (float)dim + eps);
    s.stat[0][j] = all.mean[0];
    s.stat[1][j] = rs;
    const WholePlace q = whole_place<T, TL>(tile, dim, seqlen, tiles, j / E);
    if (j % E >= q.dup) {
      if (mean_out != nullptr) mean_out[q.token + j % E] = all.mean[0];
      if (rstd_out != nullptr) rstd_out[q.token + j % E] = rs;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < E; ++k) {
    mean[k] = s.stat[0][lane % TL * E + k];
    rstd[k] = s.stat[1][lane % TL * E + k];
  }
}

// After every fourth access of a pass: memory is not accessed early across it,
// so that a pass' loads do not all claim registers at once.
__device__ __forceinline__ void hold_back(int c) {
  if ((c & 3) == 3) asm volatile("" ::: "memory");
}

}  // namespace

// A parameter of a channel: from its copy in LDS, or where the channels are too
// many for that, from global memory.
__device__ __forceinline__ float param(bool lds, const float* s, const float* p, int d) {
  return lds ? s[d] : p != nullptr ? p[d] : 0.0f;
}

// Columns, forward.  A wave takes the accesses w, w + waves, ...  The first K of
// them stay in registers from the sums to the results, `kept` more in LDS (each
// lane its own pieces); any further ones are read twice.  A workgroup fills a CU's registers, so it overlaps its own loads
// and stores: it goes over several tiles, and as a piece's result is stored the
// same registers take the next tile's piece.  weight and bias wait in LDS (a
// global load would wait for every piece in flight before it).
template <typename T, int TL, int K, bool RES>
__global__ __launch_bounds__(64 * kTileWaves, 2) void norm_cols_fwd_kernel(
    const T* __restrict__ x, const T* __restrict__ residual, const float* __restrict__ weight,
    const float* __restrict__ bias, float eps, T* __restrict__ y, T* sum_out, float* __restrict__ mean_out,
    float* __restrict__ rstd_out, int dim, int seqlen, int tiles, int all_tiles, int lds, int kept,
    int once) {
  constexpr int E = Piece<T>::kN, R = 64 / TL, U = 4;
  __shared__ TileStats<T, TL> stats;
  extern __shared__ float s_par[];  // weight, then bias, then the kept pieces
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  int first = wave * R;
  const int stride = waves * R;
  const int beyond = K * stride;  // channels held
  uint4* const s_kept = reinterpret_cast<uint4*>(s_par + (lds ? param_floats(2, dim) : 0)) + threadIdx.x;
  if (lds) {
    for (int k = threadIdx.x; k < dim; k += blockDim.x) {
      s_par[k] = weight[k];
      s_par[dim + k] = bias != nullptr ? bias[k] : 0.0f;
    }
  }
  int tile = xcd_order(blockIdx.x, gridDim.x);  // the grid has at most a workgroup per tile
  WholePlace p = whole_place<T, TL>(tile, dim, seqlen, tiles, lane);
  Piece<T> v[K];
#pragma unroll
  for (int c = 0; c < K; ++c)
    v[c] = load_whole(at_bytes(x + p.row + (int64_t)inside(first + c * stride, R, dim) * seqlen, p.at));
  for (;;) {
    first = renewed(first);
    Spread<E> sp;
    sp.clear();
    [[maybe_unused]] Piece<T> w[8];
    if constexpr (RES) {
#pragma unroll
      for (int c = 0; c < 4 && c < K; ++c)
        w[c] = load_whole(at_bytes(residual + p.row + (int64_t)inside(first + c * stride, R, dim) * seqlen, p.at));
    }
#pragma unroll
    for (int c = 0; c < K; ++c) {
      const int dw = first + c * stride, di = inside(dw, R, dim);
      const bool live = di + lane / TL >= dw;
      float f[E];
      if constexpr (RES) {
        if (c % 4 == 0) {  // the next four, four ahead
#pragma unroll
          for (int q = c + 4; q < c + 8 && q < K; ++q)
            w[q % 8] = load_whole(at_bytes(residual + p.row + (int64_t)inside(first + q * stride, R, dim) * seqlen, p.at));
        }
        float g[E];
        v[c].floats(f);
        w[c % 8].floats(g);
#pragma unroll
        for (int k = 0; k < E; ++k) f[k] += g[k];
        if (live) store_whole(at_bytes(sum_out + p.row + (int64_t)di * seqlen, p.at), p, f, false);
        v[c].set(f);  // the norm is of the stream as stored
        hold_back(c);
      }
      if (live) {
        v[c].floats(f);
        sp.add(f, 1.0f / (float)(c + 1));  // only a wave's last access is not all live
      }
#pragma unroll
      for (int k = 0; k < E; ++k) {
        settle(sp.mean[k]);
        settle(sp.sq[k]);
      }
      v[c].renew();
    }
    for (int d4 = beyond, n = 0; d4 < dim; d4 += U * stride, n += U) {  // the channels beyond
      Piece<T> e[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        e[u] = load_whole(at_bytes(x + p.row + (int64_t)inside(d4 + first + u * stride, R, dim) * seqlen, p.at));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int dw = d4 + first + u * stride, di = inside(dw, R, dim);
        if (di + lane / TL >= dw) {
          float f[E];
          e[u].floats(f);
          if constexpr (RES) {
            float g[E];
            load_whole(at_bytes(residual + p.row + (int64_t)di * seqlen, p.at)).floats(g);
#pragma unroll
            for (int k = 0; k < E; ++k) f[k] += g[k];
            store_whole(at_bytes(sum_out + p.row + (int64_t)di * seqlen, p.at), p, f, false);
            e[u].set(f);
            e[u].floats(f);
          }
          sp.add(f, rcp_hw(sp.n + 1.0f));
        }
        if (n + u < kept) keep(s_kept + (n + u) * blockDim.x, e[u]);
      }
    }
    float mean[E], rstd[E];
    tile_stats<T, TL>(sp, stats, eps, tile, dim, seqlen, tiles, mean_out, rstd_out, mean, rstd);
    first = renewed(first);
    const T* const again = RES ? sum_out : x;
    for (int d4 = beyond, n = 0; d4 < dim; d4 += U * stride, n += U) {
      Piece<T> e[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int di = inside(d4 + first + u * stride, R, dim);
        e[u] = n + u < kept ? kept_piece<T>(s_kept + (n + u) * blockDim.x)
                            : load_whole(at_bytes(again + p.row + (int64_t)di * seqlen, p.at));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int dw = d4 + first + u * stride, di = inside(dw, R, dim), d = di + lane / TL;
        if (d >= dw) {
          const float pw = param(lds, s_par, weight, d), pb = param(lds, s_par + dim, bias, d);
          float f[E];
          e[u].floats(f);
#pragma unroll
          for (int k = 0; k < E; ++k) f[k] = __builtin_fmaf((f[k] - mean[k]) * rstd[k], pw, pb);
          store_whole(at_bytes(y + p.row + (int64_t)di * seqlen, p.at), p, f, once);
        }
      }
    }
    const int next = tile + (int)gridDim.x;
    const bool more = next < all_tiles;
    const WholePlace pn = whole_place<T, TL>(more ? next : tile, dim, seqlen, tiles, lane);
#pragma unroll
    for (int c = 0; c < K; ++c) {
      const int dw = first + c * stride, di = inside(dw, R, dim), d = di + lane / TL;
      const float pw = param(lds, s_par, weight, d), pb = param(lds, s_par + dim, bias, d);
      float f[E];
      v[c].floats(f);
#pragma unroll
      for (int k = 0; k < E; ++k) f[k] = __builtin_fmaf((f[k] - mean[k]) * rstd[k], pw, pb);
      if (d >= dw) store_whole(at_bytes(y + p.row + (int64_t)di * seqlen, p.at), p, f, once);
      if (more) v[c] = load_whole(at_bytes(x + pn.row + (int64_t)di * seqlen, pn.at));
      hold_back(c);
    }
    if (!more) return;
    tile = next;
    p = pn;
  }
}

// Columns, backward: x and dy held as the forward holds x.  Writes the
// workgroup's part of dweight and dbias over its tiles, each channel's summed by
// the one lane that holds it: in LDS, or in the part itself where the channels
// are too many.
template <typename T, int TL, int K>
__global__ __launch_bounds__(64 * kTileWaves, 2) void norm_cols_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const T* __restrict__ dy, const T* __restrict__ dsum,
    T* __restrict__ dx, float* __restrict__ part, int dim, int seqlen, int tiles, int all_tiles, int lds, int kept,
    int once) {
  constexpr int E = Piece<T>::kN, R = 64 / TL, U = 2;
  __shared__ float s_part[kTileWaves][2][TL * E], s_mean[2][TL * E];
  extern __shared__ float s_par[];  // sums of dweight, of dbias, weight, then the kept pieces
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  int first = wave * R;
  const int stride = waves * R;
  const int beyond = K * stride;  // channels held
  uint4* const s_kept = reinterpret_cast<uint4*>(s_par + (lds ? param_floats(3, dim) : 0)) + threadIdx.x;
  float* const pw = part + (int64_t)blockIdx.x * 2 * dim;
  for (int k = threadIdx.x; k < dim; k += blockDim.x) {
    if (lds) {
      s_par[k] = s_par[dim + k] = 0.0f;
      s_par[2 * dim + k] = weight[k];
    } else {
      pw[k] = pw[dim + k] = 0.0f;
    }
  }
  __syncthreads();
  // one channel of an access: its steps' part of the sums over the channels
  // (s) and its own sums over the steps
  float s[2 * E], mu[E], rs[E];
  auto take = [&](const Piece<T>& px, const Piece<T>& pd, const WholePlace& p, int dw) {
    const int d = inside(dw, R, dim) + lane / TL;
    float tw = 0.0f, tb = 0.0f;
    if (d >= dw) {
      const float w = param(lds, s_par + 2 * dim, weight, d);
      float f[E], g[E];
      px.floats(f);
      pd.floats(g);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float xh = (f[k] - mu[k]) * rs[k];
        const float gw = g[k] * w;
        s[k] += gw;
        s[E + k] = __builtin_fmaf(gw, xh, s[E + k]);
        if (!p.ragged || k >= p.dup) {
          tw = __builtin_fmaf(g[k], xh, tw);
          tb += g[k];
        }
      }
    }
#pragma unroll
    for (int off = 1; off < TL; off <<= 1) {
      tw += __shfl_xor(tw, off);
      tb += __shfl_xor(tb, off);
    }
    if (d >= dw && lane % TL == 0) {
      if (lds) {
        s_par[d] += tw;
        s_par[dim + d] += tb;
      } else {
        pw[d] += tw;
        pw[dim + d] += tb;
      }
    }
#pragma unroll
    for (int k = 0; k < 2 * E; ++k) settle(s[k]);
  };
  float c1[E], c2[E];
  auto give = [&](const Piece<T>& px, const Piece<T>& pd, const WholePlace& p, int dw) {
    const int di = inside(dw, R, dim), d = di + lane / TL;
    const float w = param(lds, s_par + 2 * dim, weight, d);
    float f[E], g[E];
    px.floats(f);
    pd.floats(g);
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float xh = (f[k] - mu[k]) * rs[k];
      g[k] = rs[k] * (g[k] * w - c1[k] - xh * c2[k]);
    }
    if (dsum != nullptr) {
      load_whole(at_bytes(dsum + p.row + (int64_t)di * seqlen, p.at)).floats(f);
#pragma unroll
      for (int k = 0; k < E; ++k) g[k] += f[k];
    }
    if (d >= dw) store_whole(at_bytes(dx + p.row + (int64_t)di * seqlen, p.at), p, g, once);
  };

  int tile = xcd_order(blockIdx.x, gridDim.x);  // the grid has at most a workgroup per tile
  WholePlace p = whole_place<T, TL>(tile, dim, seqlen, tiles, lane);
  Piece<T> vx[K], vd[K];
#pragma unroll
  for (int k = 0; k < E; ++k) {
    mu[k] = mean_in[p.token + k];
    rs[k] = rstd_in[p.token + k];
  }
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int64_t base = p.row + (int64_t)inside(first + c * stride, R, dim) * seqlen;
    vx[c] = load_whole(at_bytes(x + base, p.at));
    vd[c] = load_whole(at_bytes(dy + base, p.at));
  }
  for (;;) {
    first = renewed(first);
#pragma unroll
    for (int k = 0; k < 2 * E; ++k) s[k] = 0.0f;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      take(vx[c], vd[c], p, first + c * stride);
      vx[c].renew();
      vd[c].renew();
      hold_back(c);
    }
    for (int d4 = beyond, n = 0; d4 < dim; d4 += U * stride, n += U) {  // the channels beyond
      Piece<T> ex[U], ed[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t base = p.row + (int64_t)inside(d4 + first + u * stride, R, dim) * seqlen;
        ex[u] = load_whole(at_bytes(x + base, p.at));
        ed[u] = load_whole(at_bytes(dy + base, p.at));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        take(ex[u], ed[u], p, d4 + first + u * stride);
        if (n + u < kept) {
          keep(s_kept + 2 * (n + u) * blockDim.x, ex[u]);
          keep(s_kept + (2 * (n + u) + 1) * blockDim.x, ed[u]);
        }
      }
    }
    add_lanes<TL, 2 * E>(s);
    if (lane < TL) {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        s_part[wave][0][lane * E + k] = s[k];
        s_part[wave][1][lane * E + k] = s[E + k];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * TL * E; i += blockDim.x) {
      const int q = i / (TL * E), j = i % (TL * E);
      float t = 0.0f;
      for (int w = 0; w < waves; ++w) t += s_part[w][q][j];
      s_mean[q][j] = t / (float)dim;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < E; ++k) {
      c1[k] = s_mean[0][lane % TL * E + k];
      c2[k] = s_mean[1][lane % TL * E + k];
    }
    first = renewed(first);
    for (int d4 = beyond, n = 0; d4 < dim; d4 += U * stride, n += U) {
      Piece<T> ex[U], ed[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t base = p.row + (int64_t)inside(d4 + first + u * stride, R, dim) * seqlen;
        if (n + u < kept) {
          ex[u] = kept_piece<T>(s_kept + 2 * (n + u) * blockDim.x);
          ed[u] = kept_piece<T>(s_kept + (2 * (n + u) + 1) * blockDim.x);
        } else {
          ex[u] = load_whole(at_bytes(x + base, p.at));
          ed[u] = load_whole(at_bytes(dy + base, p.at));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) give(ex[u], ed[u], p, d4 + first + u * stride);
    }
    const int next = tile + (int)gridDim.x;
    const bool more = next < all_tiles;
    const WholePlace pn = whole_place<T, TL>(more ? next : tile, dim, seqlen, tiles, lane);
    float mun[E], rsn[E];
#pragma unroll
    for (int k = 0; k < E; ++k) {
      mun[k] = mean_in[pn.token + k];
      rsn[k] = rstd_in[pn.token + k];
    }
#pragma unroll
    for (int c = 0; c < K; ++c) {
      give(vx[c], vd[c], p, first + c * stride);
      if (more) {
        const int64_t base = pn.row + (int64_t)inside(first + c * stride, R, dim) * seqlen;
        vx[c] = load_whole(at_bytes(x + base, pn.at));
        vd[c] = load_whole(at_bytes(dy + base, pn.at));
      }
      hold_back(c);
    }
    if (!more) break;
    tile = next;
    p = pn;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      mu[k] = mun[k];
      rs[k] = rsn[k];
    }
  }
  if (lds) {
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * dim; k += blockDim.x) pw[k] = s_par[k];
  }
}

// Columns of fewer steps than a piece (under 16 bytes a row): a workgroup per
// token, its threads over the channels.
template <typename T>
__global__ __launch_bounds__(256) void norm_few_fwd_kernel(
    const T* __restrict__ x, const T* __restrict__ residual, const float* __restrict__ weight,
    const float* __restrict__ bias, float eps, T* __restrict__ y, T* sum_out, float* __restrict__ mean_out,
    float* __restrict__ rstd_out, int64_t tokens, int dim, int seqlen) {
  __shared__ double s_mean[4][kMaxRowWaves];
  __shared__ float s_var[4][kMaxRowWaves];
  const int64_t token = group_index();
  if (token >= tokens) return;
  const int wave = threadIdx.x >> 6;
  const int64_t base = token / seqlen * dim * seqlen + token % seqlen;
  const T* const again = residual != nullptr ? sum_out : x;
  double sum = 0.0;
  for (int d = threadIdx.x; d < dim; d += 256) {
    const int64_t at = base + (int64_t)d * seqlen;
    float f = Elem<T>::load(x + at);
    if (residual != nullptr) {
      f += Elem<T>::load(residual + at);
      Elem<T>::store(sum_out + at, f);
      f = Elem<T>::load(sum_out + at);  // the norm is of the stream as stored
    }
    sum += f;
  }
  const float mean = (float)(row_sum(sum, s_mean, 0, wave, 4) / (double)dim);
  float sq = 0.0f;
  for (int d = threadIdx.x; d < dim; d += 256) {
    const float f = Elem<T>::load(again + base + (int64_t)d * seqlen) - mean;
    sq = __builtin_fmaf(f, f, sq);
  }
  const float rstd = 1.0f / __builtin_sqrtf(row_sum(sq, s_var, 0, wave, 4) / (float)dim + eps);
  if (threadIdx.x == 0) {
    if (mean_out != nullptr) mean_out[token] = mean;
    if (rstd_out != nullptr) rstd_out[token] = rstd;
  }
  for (int d = threadIdx.x; d < dim; d += 256) {
    const int64_t at = base + (int64_t)d * seqlen;
    Elem<T>::store(y + at, __builtin_fmaf((Elem<T>::load(again + at) - mean) * rstd, weight[d],
                                          bias != nullptr ? bias[d] : 0.0f));
  }
}

// dx, and the workgroup's part of dweight and dbias over its tokens (its own,
// then every gridDim.x-th), one token at a time: each thread its channels.
template <typename T>
__global__ __launch_bounds__(256) void norm_few_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const T* __restrict__ dy, const T* __restrict__ dsum,
    T* __restrict__ dx, float* __restrict__ part, int64_t tokens, int dim, int seqlen) {
  __shared__ float s_a[2][4][kMaxRowWaves], s_b[2][4][kMaxRowWaves];
  float* const pw = part + (int64_t)blockIdx.x * 2 * dim;
  const int wave = threadIdx.x >> 6;
  const float n = (float)dim;
  int turn = 0;
  for (int64_t token = blockIdx.x; token < tokens; token += gridDim.x, turn ^= 1) {
    const bool begin = token == blockIdx.x;
    const int64_t base = token / seqlen * dim * seqlen + token % seqlen;
    const float mu = mean_in[token], rs = rstd_in[token];
    float c1 = 0.0f, c2 = 0.0f;
    for (int d = threadIdx.x; d < dim; d += 256) {
      const int64_t at = base + (int64_t)d * seqlen;
      const float xh = (Elem<T>::load(x + at) - mu) * rs, g = Elem<T>::load(dy + at);
      pw[d] = begin ? g * xh : __builtin_fmaf(g, xh, pw[d]);
      pw[dim + d] = begin ? g : pw[dim + d] + g;
      c1 = __builtin_fmaf(g, weight[d], c1);
      c2 = __builtin_fmaf(g * weight[d], xh, c2);
    }
    c1 = row_sum(c1, s_a[turn], 0, wave, 4) / n;
    c2 = row_sum(c2, s_b[turn], 0, wave, 4) / n;
    for (int d = threadIdx.x; d < dim; d += 256) {
      const int64_t at = base + (int64_t)d * seqlen;
      const float xh = (Elem<T>::load(x + at) - mu) * rs;
      const float v = rs * (Elem<T>::load(dy + at) * weight[d] - c1 - xh * c2);
      Elem<T>::store(dx + at, dsum != nullptr ? v + Elem<T>::load(dsum + at) : v);
    }
  }
}

// dweight[d] = sum_p part[p][0][d], dbias[d] = sum_p part[p][1][d].  A
// workgroup takes 32 of the 2 dim sums, 32 threads each.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* __restrict__ part, float* __restrict__ dweight,
                                                        float* __restrict__ dbias, int parts, int dim) {
  __shared__ float s[32][33];
  const int64_t at = group_index() * 32 + (threadIdx.x & 31);
  const int j = threadIdx.x >> 5;
  float v = 0.0f;
  if (at < 2 * (int64_t)dim) {
    constexpr int U = 8;  // loads in flight
    int p = j;
    for (; p + 32 * (U - 1) < parts; p += 32 * U) {
      float f[U];
#pragma unroll
      for (int u = 0; u < U; ++u) f[u] = part[(int64_t)(p + 32 * u) * 2 * dim + at];
#pragma unroll
      for (int u = 0; u < U; ++u) v += f[u];
    }
    for (; p < parts; p += 32) v += part[(int64_t)p * 2 * dim + at];
  }
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

// Rows: lanes of a row shorter than a wave (8, 16, 32; else 64), waves of a row,
// accesses of a lane (1, 2 or 4; 0: a row too long for a workgroup's registers).
struct RowPlan {
  int LR, W, K;
  int lanes() const { return LR < 64 ? LR : 64 * W; }
};

// `least`: accesses of a lane where a row has that many (the 16-bit forward's, see
// rows_fwd_plan).
RowPlan row_plan(int dim, int least = 1) {
  for (int LR = 8; LR < 64; LR *= 2)
    if (dim <= LR * kRun) return RowPlan{LR, 1, 1};
  const int spans = (dim + kRowSpan - 1) / kRowSpan;
  int K = spans < least ? 1 : least;
  while (K < 4 && spans > kMaxRowWaves * K) K *= 2;
  if (spans > kMaxRowWaves * K) return RowPlan{64, 0, 0};
  return RowPlan{64, (spans + K - 1) / K, K};
}

// The forward holds nothing over its rows, and a wave waits on its own few loads:
// of 16-bit types two accesses a lane (32768 rows of 2560 bf16: 72 us, with one 88,
// with four 74; with a residual 119, 140, 134; 16384 rows of 1000: 13, 15, 19),
// of float32, whose access is twice as long, one (128, 126 and 129; with a
// residual 258, 242, 256).  Fewer, longer-lived workgroups that read their next
// row ahead were no faster (88 us and more).  Also for few rows, where one is
// quicker (256 rows of 2560 with a residual: 3.8 us, two 4.6): a token's sums are
// then in one order, and its result the same bits, in a batch of any size.  The
// backward's sums of dweight and dbias want the registers (16384 rows of 2560: one
// access 74 us, two 88).
template <typename T>
RowPlan rows_fwd_plan(int dim) { return row_plan(dim, sizeof(T) == 2 ? 2 : 1); }

// The backward's workgroups: several short rows (their sums of dweight and dbias
// then make one part) or a long one, and 4 rows and more to a slot, so that the
// parts stay small beside the rows (16384 rows of 2560 bf16: 512 workgroups 88
// us, 768 78, 1024 81; of 1000: 33, 35, 37).
int row_bwd_slots(const RowPlan& pl) { return pl.lanes() <= 128 ? 512 / pl.lanes() : 1; }

int row_bwd_groups(const RowPlan& pl, int rows) {
  const int64_t per = 4 * (int64_t)row_bwd_slots(pl);
  const int64_t g = (rows + per - 1) / per;
  const int most = pl.lanes() <= 128 ? 512 : 768;
  return (int)(g < most ? g : most);
}

// Columns: lanes of a channel's piece (0: fewer steps than a piece), accesses a
// wave holds in registers, waves of a workgroup, tiles of a batch row and of the
// call, workgroups, LDS for parameters and kept accesses.
struct ColPlan {
  int TL, K, waves, tiles, all, groups;
  size_t room;
};

// What a column kernel holds: accesses in registers (the first two with half a CU's
// LDS, the last with the registers and LDS of a CU to one workgroup), most
// workgroups, parameters (and sums of their gradients) a channel and the most
// channels for which they wait in LDS, arrays that it holds pieces of.
// Workgroups: the forward's are two for each CU (batch 16, dim 5120, L 2048 bf16:
// 164 us, with one 170).  The backward's each leave a part of dweight and dbias, so
// one for each CU, whatever it holds (batch 8, dim 1536, L 2047 float32: 88 us, with
// two 97); its smaller plan, which in bf16 builds to 129 registers and could not run
// twice on a CU, is there for what needs no more (batch 8, L 2048 bf16: dim 500 17 us,
// 768 27, 1536 39).
struct ColKind {
  int held[3], groups, params, lds_dim, arrays;
};

constexpr ColKind kColFwd = {{10, 16, 40}, 512, 2, 8192, 1};
constexpr ColKind kColSum = {{10, 10, 20}, 512, 2, 8192, 1};  // forward with a residual
constexpr ColKind kColBwd = {{5, 5, 16}, 256, 3, 5120, 2};

// Dynamic LDS of a column kernel: the parameters, then accesses that the registers
// do not hold, as far as the plan's room goes.
struct LdsPlan {
  int lds, kept;
  size_t bytes;
};

LdsPlan lds_plan(const ColKind& kind, const ColPlan& p, int dim) {
  LdsPlan l{};
  l.lds = dim <= kind.lds_dim;
  l.bytes = l.lds ? (size_t)param_floats(kind.params, dim) * 4 : 0;
  const int rows = 64 / p.TL, need = (dim + rows - 1) / rows;
  const int each = (need + p.waves - 1) / p.waves;  // accesses of a wave
  const size_t access = (size_t)p.waves * 64 * 16 * kind.arrays;
  if (each > p.K && p.TL < 64 && p.room > l.bytes) {  // (of TL = 64 the sums' arrays are too long)
    const size_t fit = (p.room - l.bytes) / access;
    l.kept = each - p.K < (int)fit ? each - p.K : (int)fit;
    l.bytes += (size_t)l.kept * access;
  }
  return l;
}

ColPlan col_plan(const ColKind& kind, int batch, int dim, int64_t seqlen, int elem_bytes) {
  ColPlan p{};
  const int64_t row = seqlen * elem_bytes;
  if (row < 16 || row >= INT32_MAX) {
    const int64_t tokens = (int64_t)batch * seqlen;
    p.groups = (int)(tokens < 512 ? tokens : 512);
    return p;
  }
  // Whole lines of 128 bytes where they make enough tiles for the chip (batch
  // 16, dim 5120, L 2048 bf16, the tiles' pattern alone as a copy: 256 bytes 131
  // us, 128 bytes 145, 64 bytes 207, 32 bytes 368); fewer channels than an
  // access has: one channel an access.
  p.TL = 8;
  while (p.TL > 1 && (int64_t)batch * ((row + 16 * p.TL - 1) / (16 * p.TL)) < 256) p.TL /= 2;
  while (dim < 64 / p.TL) p.TL = p.TL < 8 ? 2 * p.TL : 64;
  if (row * (64 / p.TL) >= INT32_MAX) p.TL = 64;  // byte offsets within an access in 32 bits
  const int need = (dim + 64 / p.TL - 1) / (64 / p.TL);
  p.waves = need < kTileWaves ? need : kTileWaves;
  p.tiles = (int)((row + 16 * p.TL - 1) / (16 * p.TL));
  p.all = batch * p.tiles;
  p.groups = p.all < kind.groups ? p.all : kind.groups;
  // A CU's 160 KiB of LDS, or half of them, less the sums' static arrays.  Two
  // workgroups of a CU overlap one's loads with the other's stores, so the forward
  // takes them as long as they hold all but an access of a wave (batch 16, L 2048
  // bf16, dim 768: 20 us, one workgroup with 40 accesses held 35).
  const int each = (need + p.waves - 1) / p.waves;
  p.room = (size_t)75 * 1024;
  for (int k = 0; k < 2; ++k) {
    p.K = kind.held[k];
    if (each <= p.K + lds_plan(kind, p, dim).kept + (k == 1 ? 1 : 0)) return p;
  }
  p.K = kind.held[2];
  p.room = (size_t)155 * 1024;
  return p;
}

// Whether every access writes whole lines of `out`.
int whole_lines(const NormLaunch& a, const ColPlan& p, size_t es, const void* out) {
  return p.TL >= 8 && (size_t)a.seqlen * es % 128 == 0 && reinterpret_cast<uintptr_t>(out) % 128 == 0;
}

template <typename T, int K, int LR>
hipError_t rows_fwd(const NormLaunch& a, const RowPlan& pl, hipStream_t stream) {
  const int slots = pl.lanes() < 256 ? 256 / pl.lanes() : 1;
  const dim3 grid = grid_of(((int64_t)a.batch + slots - 1) / slots, pl.lanes() * slots);
  norm_rows_fwd_kernel<T, K, LR><<<grid, pl.lanes() * slots, 0, stream>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.residual), a.weight, a.bias, a.eps,
      static_cast<T*>(a.y), static_cast<T*>(a.sum_out), a.mean, a.rstd, a.batch, a.dim, 1.0 / a.dim, pl.W);
  return hipGetLastError();
}

template <typename T, int K, int LR>
hipError_t rows_bwd(const NormLaunch& a, const RowPlan& pl, hipStream_t stream) {
  const int slots = row_bwd_slots(pl);
  norm_rows_bwd_kernel<T, K, LR><<<(unsigned)row_bwd_groups(pl, a.batch), pl.lanes() * slots,
                                   slots > 1 ? (size_t)a.dim * 8 * slots : 0, stream>>>(
      static_cast<const T*>(a.x), a.weight, a.mean, a.rstd, static_cast<const T*>(a.dy),
      static_cast<const T*>(a.dsum), static_cast<T*>(a.dx), a.part, a.batch, a.dim, pl.W);
  return hipGetLastError();
}

// f<K, LR> of a row plan.
template <typename F>
hipError_t by_row_plan(const RowPlan& pl, F&& f) {
  switch (pl.LR) {
    case 8: return f.template operator()<1, 8>();
    case 16: return f.template operator()<1, 16>();
    case 32: return f.template operator()<1, 32>();
  }
  return pl.K == 1 ? f.template operator()<1, 64>()
                   : pl.K == 2 ? f.template operator()<2, 64>() : f.template operator()<4, 64>();
}

template <typename T>
struct RowsFwd {
  const NormLaunch& a;
  const RowPlan& pl;
  hipStream_t stream;
  template <int K, int LR>
  hipError_t operator()() const { return rows_fwd<T, K, LR>(a, pl, stream); }
};

template <typename T>
struct RowsBwd {
  const NormLaunch& a;
  const RowPlan& pl;
  hipStream_t stream;
  template <int K, int LR>
  hipError_t operator()() const { return rows_bwd<T, K, LR>(a, pl, stream); }
};

template <typename T, int TL, int K, bool RES>
hipError_t cols_fwd_launch(const NormLaunch& a, const ColPlan& p, hipStream_t stream) {
  const LdsPlan l = lds_plan(RES ? kColSum : kColFwd, p, a.dim);
  norm_cols_fwd_kernel<T, TL, K, RES><<<(unsigned)p.groups, 64 * p.waves, l.bytes, stream>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.residual), a.weight, a.bias, a.eps,
      static_cast<T*>(a.y), static_cast<T*>(a.sum_out), a.mean, a.rstd, a.dim, (int)a.seqlen, p.tiles, p.all, l.lds, l.kept,
      whole_lines(a, p, sizeof(T), a.y));
  return hipGetLastError();
}

template <typename T, int TL>
hipError_t cols_fwd(const NormLaunch& a, const ColPlan& p, hipStream_t stream) {
  constexpr const int (&fwd)[3] = kColFwd.held, (&sum)[3] = kColSum.held;
  if (a.residual != nullptr)
    return p.K == sum[2] ? cols_fwd_launch<T, TL, sum[2], true>(a, p, stream)
                         : cols_fwd_launch<T, TL, sum[0], true>(a, p, stream);
  return p.K == fwd[2]   ? cols_fwd_launch<T, TL, fwd[2], false>(a, p, stream)
         : p.K == fwd[1] ? cols_fwd_launch<T, TL, fwd[1], false>(a, p, stream)
                         : cols_fwd_launch<T, TL, fwd[0], false>(a, p, stream);
}

template <typename T, int TL>
hipError_t cols_bwd(const NormLaunch& a, const ColPlan& p, hipStream_t stream) {
  const LdsPlan l = lds_plan(kColBwd, p, a.dim);
  constexpr const int (&held)[3] = kColBwd.held;
  auto kernel = p.K == held[2] ? norm_cols_bwd_kernel<T, TL, held[2]> : norm_cols_bwd_kernel<T, TL, held[0]>;
  kernel<<<(unsigned)p.groups, 64 * p.waves, l.bytes, stream>>>(
      static_cast<const T*>(a.x), a.weight, a.mean, a.rstd, static_cast<const T*>(a.dy),
      static_cast<const T*>(a.dsum), static_cast<T*>(a.dx), a.part, a.dim, (int)a.seqlen, p.tiles, p.all, l.lds, l.kept,
      whole_lines(a, p, sizeof(T), a.dx));
  return hipGetLastError();
}

template <typename T>
hipError_t fwd_typed(const NormLaunch& a, hipStream_t stream) {
  const RowPlan pl = rows_fwd_plan<T>(a.dim);
  if (a.seqlen == 1 && pl.K > 0) return by_row_plan(pl, RowsFwd<T>{a, pl, stream});
  const ColPlan cp = col_plan(a.residual != nullptr ? kColSum : kColFwd, a.batch, a.dim, a.seqlen, sizeof(T));
  switch (cp.TL) {
    case 1: return cols_fwd<T, 1>(a, cp, stream);
    case 2: return cols_fwd<T, 2>(a, cp, stream);
    case 4: return cols_fwd<T, 4>(a, cp, stream);
    case 8: return cols_fwd<T, 8>(a, cp, stream);
    case 64: return cols_fwd<T, 64>(a, cp, stream);
  }
  const int64_t tokens = (int64_t)a.batch * a.seqlen;
  norm_few_fwd_kernel<T><<<grid_of(tokens, 256), 256, 0, stream>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.residual), a.weight, a.bias, a.eps,
      static_cast<T*>(a.y), static_cast<T*>(a.sum_out), a.mean, a.rstd, tokens, a.dim, (int)a.seqlen);
  return hipGetLastError();
}

template <typename T>
hipError_t bwd_typed(const NormLaunch& a, hipStream_t stream) {
  const RowPlan pl = row_plan(a.dim);
  hipError_t e;
  if (a.seqlen == 1 && pl.K > 0) {
    e = by_row_plan(pl, RowsBwd<T>{a, pl, stream});
  } else {
    const ColPlan cp = col_plan(kColBwd, a.batch, a.dim, a.seqlen, sizeof(T));
    switch (cp.TL) {
      case 1: e = cols_bwd<T, 1>(a, cp, stream); break;
      case 2: e = cols_bwd<T, 2>(a, cp, stream); break;
      case 4: e = cols_bwd<T, 4>(a, cp, stream); break;
      case 8: e = cols_bwd<T, 8>(a, cp, stream); break;
      case 64: e = cols_bwd<T, 64>(a, cp, stream); break;
      default:
        norm_few_bwd_kernel<T><<<(unsigned)cp.groups, 256, 0, stream>>>(
            static_cast<const T*>(a.x), a.weight, a.mean, a.rstd, static_cast<const T*>(a.dy),
            static_cast<const T*>(a.dsum), static_cast<T*>(a.dx), a.part, (int64_t)a.batch * a.seqlen, a.dim,
            (int)a.seqlen);
        e = hipGetLastError();
    }
  }
  if (e != hipSuccess) return e;
  const int parts = norm_bwd_parts(a.batch, a.dim, a.seqlen, sizeof(T));
  norm_sum_kernel<<<grid_of((2 * (int64_t)a.dim + 31) / 32, 1024), 1024, 0, stream>>>(a.part, a.dweight, a.dbias,
                                                                                   parts, a.dim);
  return hipGetLastError();
}

}  // namespace

int norm_bwd_parts(int batch, int dim, int64_t seqlen, int elem_bytes) {
  const RowPlan pl = row_plan(dim);
  if (seqlen == 1 && pl.K > 0) return row_bwd_groups(pl, batch);
  return col_plan(kColBwd, batch, dim, seqlen, elem_bytes).groups;
}

hipError_t launch_norm_fwd(const NormLaunch& a, hipStream_t stream) {
  return a.dtype == Dtype::BF16 ? fwd_typed<uint16_t>(a, stream) : fwd_typed<float>(a, stream);
}

hipError_t launch_norm_bwd(const NormLaunch& a, hipStream_t stream) {
  return a.dtype == Dtype::BF16 ? bwd_typed<uint16_t>(a, stream) : bwd_typed<float>(a, stream);
}

}  // namespace ssm
