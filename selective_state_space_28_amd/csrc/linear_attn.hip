// linear_attn.hip -- linear attention with a decay for each head, for gfx950
// (include/ssm_linear_attn.h states it): the chunked sweep that the forward pass
// and every gradient are made of, the decay's gradient, and the single token.
//
// With W_ij = e^{g (i-j)} for j <= i, a chunk of C steps that the state S enters is
//
//   O  = (W o Q K^T) V + diag(e^{g (i+1)}) Q S        (C x C products, then C x kd x vd)
//   S <- e^{g C} S + (diag(e^{g (C-1-j)}) K)^T V       (kd x C x vd)
//
// and the gradients are the same sweep with its operands in other places:
//
//   dq:  q <- dy, k <- v,  v <- k,  S transposed        forward in time
//   dk:  q <- v,  k <- dy, v <- q,  dS transposed       backward in time
//   dv:  q <- k,  k <- q,  v <- dy, dS                  backward in time
//
// where backward in time the state is passed on already decayed (dS_t of the
// state *before* step t's decay is what the step before receives): the entering
// weights are e^{g i} and the leaving ones e^{g (C-j)} (`sh` below).
//
// A workgroup owns a (batch row, head, segment) and 16 value columns for each of
// its waves.  S never leaves the matrix cores' accumulators.  16-bit operands use
// v_mfma_f32_16x16x32_bf16, float32 v_mfma_f32_16x16x4_f32.
#include "linear_attn.hpp"
#include "runs.hpp"
#include "ssm_math.hpp"

namespace ssm {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ bool finite_f32(float v) { return __builtin_fabsf(v) <= 3.4028234664e38f; }

// e^{g n} of n >= 0 steps, held at or above the smallest normal float where one
// step's decay is (an infinite state stays infinite, and 0 inf is not formed); the
// product's and the conversion's roundings are carried along, since the exponent
// of many steps is large.  n = 0: 1, whatever g is.
__device__ __forceinline__ float decay_pow(float g, float n) {
  if (n == 0.0f) return 1.0f;
  const float p = g * n;
  float v;
  if (__builtin_fabsf(p) < 200.0f) {
    constexpr float kLog2eLow = 1.925963033500234e-8f;  // log2 e - kLog2e
    const float plow = __builtin_fmaf(g, n, -p);
    const float hi = p * kLog2e;
    const float low = __builtin_fmaf(p, kLog2e, -hi) + __builtin_fmaf(p, kLog2eLow, plow * kLog2e);
    v = exp2_hw(hi) * __builtin_fmaf(low, kLn2, 1.0f);
  } else {
    v = exp2_hw(p * kLog2e);
  }
  return g > -87.0f && v < kMinNormal ? kMinNormal : v;
}

// The matrix cores' operands for storage type T.  A fragment is what a lane
// supplies of CK contracted elements: with q = lane / 16, m = lane % 16, of row (or
// column) m the elements 8 q + e of 32 (bf16, e < 8) or 4 q + e of 16 (float32,
// e < 4, four products).  A product's lane receives D[4 q + r][m], r < 4.
template <typename T>
struct Mat;

template <>
struct Mat<uint16_t> {
  static constexpr int C = 64;    // steps of a chunk
  static constexpr int CK = 32;
  static constexpr int E = 8;     // elements of a fragment
  static constexpr int kPad = 8;  // elements behind a row in LDS
  typedef bf16x8 Frag;
  __device__ __forceinline__ static f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // of a row-major tile, contracted along its rows
  __device__ __forceinline__ static Frag row(const uint16_t* tile, int ld, int r0, int c0, int lane) {
    return *reinterpret_cast<const Frag*>(tile + (r0 + (lane & 15)) * ld + c0 + 8 * (lane >> 4));
  }
  // the same, in the order in which the accumulators hold S: 4 q + r of the first 16, then of the second
  __device__ __forceinline__ static Frag row_as_state(const uint16_t* tile, int ld, int r0, int c0, int lane) {
    const uint16_t* p = tile + (r0 + (lane & 15)) * ld + c0 + 4 * (lane >> 4);
    const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(p + 16);
    return __builtin_bit_cast(Frag, make_uint4(a.x, a.y, b.x, b.y));
  }
  // contracted along its columns: the transposing LDS read gives 4 rows of a column to a lane
  __device__ __forceinline__ static Frag col(const uint16_t* tile, int ld, int r0, int c0, int lane) {
    const uint16_t* p = tile + (r0 + 8 * (lane >> 4) + ((lane & 15) >> 2)) * ld + c0 + 4 * (lane & 3);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * ld));
    const s16x4 ab[2] = {a, b};
    return __builtin_bit_cast(Frag, ab);
  }
  __device__ __forceinline__ static float at(const Frag& f, int e) { return (float)f[e]; }
  __device__ __forceinline__ static void zero(Frag& f, int e) { f[e] = (__bf16)0.0f; }
};

template <>
struct Mat<float> {
  static constexpr int C = 32;
  static constexpr int CK = 16;
  static constexpr int E = 4;
  static constexpr int kPad = 4;
  typedef f32x4 Frag;
  __device__ __forceinline__ static f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
  }
  __device__ __forceinline__ static Frag row(const float* tile, int ld, int r0, int c0, int lane) {
    return *reinterpret_cast<const Frag*>(tile + (r0 + (lane & 15)) * ld + c0 + 4 * (lane >> 4));
  }
  __device__ __forceinline__ static Frag row_as_state(const float* tile, int ld, int r0, int c0, int lane) {
    return row(tile, ld, r0, c0, lane);
  }
  __device__ __forceinline__ static Frag col(const float* tile, int ld, int r0, int c0, int lane) {
    const float* p = tile + (r0 + 4 * (lane >> 4)) * ld + c0 + (lane & 15);
    return Frag{p[0], p[ld], p[2 * ld], p[3 * ld]};
  }
  __device__ __forceinline__ static float at(const Frag& f, int e) { return f[e]; }
  __device__ __forceinline__ static void zero(Frag& f, int e) { f[e] = 0.0f; }
};

// A float32 as a sum of N bf16 fragments' elements: the leading bits cut off, what
// is left cut off again, the last rounded.  Three hold a float32 exactly, two to
// 2^-16.  (Of an infinite value the rest is NaN, and so is what it meets.)
__device__ __forceinline__ float cut16(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

template <typename T, int N>
struct Parts {
  typename Mat<T>::Frag f[N];
};

template <int N>
__device__ __forceinline__ Parts<uint16_t, N> parts_of(const float (&x)[8]) {
  Parts<uint16_t, N> p;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float v = x[e];
#pragma unroll
    for (int k = 0; k < N - 1; ++k) {
      const float hi = cut16(v);
      p.f[k][e] = (__bf16)hi;
      v -= hi;
    }
    p.f[N - 1][e] = (__bf16)v;
  }
  return p;
}

template <int N>
__device__ __forceinline__ Parts<float, 1> parts_of(const float (&x)[4]) {
  Parts<float, 1> p;
  p.f[0] = f32x4{x[0], x[1], x[2], x[3]};
  return p;
}

// ---- staging ----------------------------------------------------------------------
// Rows u0 .. u0 + C of a (batch, head) slice into LDS, `WIDTH` columns: zeros from
// column `width` and from row n on.  Step u is at row base + u * st (st < 0 backward
// in time).
template <typename T, int ROWS, int WIDTH, int LD, int THREADS>
__device__ __forceinline__ void stage(T* lds, const T* base, int64_t st, int width, int n, bool vec) {
  constexpr int VE = 16 / (int)sizeof(T);
  constexpr int kPerRow = WIDTH / VE;
  for (int i = threadIdx.x; i < ROWS * kPerRow; i += THREADS) {
    const int r = i / kPerRow, c = (i % kPerRow) * VE;
    const T* p = base + r * st + c;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (r < n && c < width) {
      if (vec && c + VE <= width) {
        w = *reinterpret_cast<const uint4*>(p);
      } else {
        T e[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k) e[k] = c + k < width ? p[k] : (T)0;
        __builtin_memcpy(&w, e, 16);
      }
    }
    *reinterpret_cast<uint4*>(lds + r * LD + c) = w;
  }
}

}  // namespace

enum AttnMode { kAttnOut = 0, kAttnSegments = 1, kAttnDecay = 2 };

// One workgroup: NW waves, 16 value columns each.  kAttnSegments: only the state that
// a segment adds, and what it leaves of the one before.  kAttnDecay: the forward
// sweep with R = dS/dg beside S, and dg = scale sum_t q_t R_t dy_t + <R_L, dlast>;
// R_u = e^g (R_{u-1} + S_{u-1}) gives, of a chunk,
//   diag(e^{g (i+1)}) Q (R + (i+1) S) + ((i-j) W o Q K^T) V
//   R <- e^{g C} (R + C S) + (diag((C-1-j) e^{g (C-1-j)}) K)^T V
template <typename T, int KD, int NW, int MODE>
__global__ __launch_bounds__(64 * NW) void attn_sweep_kernel(const AttnSweep a, const float* __restrict__ dlast) {
  using M = Mat<T>;
  using Frag = typename M::Frag;
  constexpr int C = M::C, IT = C / 16, CK = M::CK, E = M::E;
  constexpr int NV = 16 * NW, THREADS = 64 * NW;
  constexpr int LDK = KD + M::kPad, LDV = NV + M::kPad, LDP = C + M::kPad;
  constexpr int KT = KD / 16;  // tiles of S in a wave
  constexpr bool kDecay = MODE == kAttnDecay, kOut = MODE != kAttnSegments;
  constexpr int NU = sizeof(T) == 2 ? 3 : 1;  // parts of the decayed v, exact
  constexpr int NS = sizeof(T) == 2 ? 2 : 1;  // parts of S as an operand, to 2^-16

  __shared__ __attribute__((aligned(16))) T s_q[kOut ? C * LDK : 1];
  __shared__ __attribute__((aligned(16))) T s_k[C * LDK];
  __shared__ __attribute__((aligned(16))) T s_v[C * LDV];
  __shared__ __attribute__((aligned(16))) T s_p[kOut ? C * LDP : 1];
  __shared__ __attribute__((aligned(16))) T s_p2[kDecay && sizeof(T) == 2 ? C * LDP : 1];  // second parts
  __shared__ __attribute__((aligned(16))) T s_dy[kDecay ? C * LDV : 1];
  __shared__ float s_pw[C + 1];
  __shared__ double s_sum[NW];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, q4 = 4 * (lane >> 4);
  const int nvb = (a.vd + NV - 1) / NV;
  const int nsegs = MODE == kAttnSegments ? a.nseg - 1 : MODE == kAttnDecay ? 1 : a.nseg;
  int64_t id = group_index();
  if (id >= (int64_t)a.batch * a.heads * nvb * nsegs) return;
  const int vb = (int)(id % nvb);
  id /= nvb;
  const int h = (int)(id % a.heads);
  id /= a.heads;
  const int seg = (int)(id % nsegs), b = (int)(id / nsegs);

  const float g = a.g[h];
  const int L = (int)a.seqlen;
  const int len = a.lengths == nullptr ? L : min(max(a.lengths[b], 0), L);
  const int sh = a.rev ? 1 : 0;
  for (int i = threadIdx.x; i <= C; i += THREADS) s_pw[i] = decay_pow(g, (float)i);

  const int v0 = vb * NV;                     // first value column of the workgroup
  const int vw = min(NV, a.vd - v0);          // its columns
  const int col = v0 + 16 * wave + m;         // of S, this lane's
  const int64_t head = (int64_t)b * a.heads + h;
  const int64_t dir = a.rev ? -1 : 1, first = a.rev ? len - 1 : 0;
  const auto base = [&](const AttnView& w) {
    return static_cast<const T*>(w.p) + b * w.sb + (h / w.share) * w.sh + first * w.st;
  };
  const T *pq = base(a.q), *pk = base(a.k), *pv = base(a.v) + v0, *pdy = kDecay ? base(a.dy) + v0 : nullptr;
  const auto vectors = [](const AttnView& w, int width) {
    constexpr int VE = 16 / (int)sizeof(T);
    return reinterpret_cast<uintptr_t>(w.p) % 16 == 0 && ((w.sb | w.st | w.sh | (int64_t)width) % VE) == 0;
  };
  const bool vec_q = vectors(a.q, 0), vec_k = vectors(a.k, 0), vec_v = vectors(a.v, 0),
             vec_dy = kDecay && vectors(a.dy, 0);

  // S: rows 16 t + q4 + r, column `col`
  f32x4 S[KT], R[kDecay ? KT : 1];
#pragma unroll
  for (int t = 0; t < KT; ++t) {
    if constexpr (kDecay) R[t] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * t + q4 + r;
      float v = 0.0f;
      if (kOut && row < a.kd && col < a.vd) {
        const int64_t mat = (int64_t)a.kd * a.vd;
        if (seg > 0)
          v = a.seg_state[(head * a.nseg + seg) * mat + (int64_t)row * a.vd + col];
        else if (a.state_in != nullptr)
          v = a.state_in[head * mat + (a.transposed ? (int64_t)col * a.kd + row : (int64_t)row * a.vd + col)];
      }
      S[t][r] = v;
    }
  }
  if constexpr (kOut) {  // the masked halves of pairs of tiles stay zero
    for (int i = threadIdx.x; i < C * LDP; i += THREADS) {
      s_p[i] = (T)0;
      if constexpr (kDecay && sizeof(T) == 2) s_p2[i] = (T)0;
    }
  }
  double dg = 0.0;
  float through = 1.0f;  // kAttnSegments: of the whole segment
  bool cut = false;

  const int u_begin = (int)(seg * a.seglen);
  const int u_end = MODE == kAttnDecay ? L : (int)min((int64_t)L, u_begin + a.seglen);
  T* out = static_cast<T*>(a.out);
  for (int u0 = u_begin; u0 < u_end; u0 += C) {
    const int n = min(max(len - u0, 0), C);
    if (n == 0 && MODE != kAttnOut) break;
    if (kOut && n == 0) {  // steps behind the row's length
      for (int64_t i = threadIdx.x; i < (int64_t)(u_end - u0) * vw; i += THREADS) {
        const int64_t at = (((int64_t)b * L + u0 + i / vw) * a.heads + h) * a.vd + v0 + i % vw;
        if (a.out_f32) static_cast<float*>(a.out)[at] = 0.0f;
        else out[at] = (T)0;
      }
      break;
    }
    // bit i: no state and no product crosses from step i-1 to step i
    uint64_t B = 0;
    if (a.starts != nullptr) {
      const int u = u0 + lane;
      bool f = false;
      if (lane < n && !(a.rev && u == 0)) f = a.starts[(int64_t)b * L + (a.rev ? len - u : u)] != 0;
      B = __ballot(f);
    }
    const auto seen = [&](int i) { return __popcll(B & (~0ull >> (63 - i))); };  // starts up to and with step i

    __syncthreads();  // the chunk before is done with LDS
    if constexpr (kOut) stage<T, C, KD, LDK, THREADS>(s_q, pq + u0 * dir * a.q.st, dir * a.q.st, a.kd, n, vec_q);
    stage<T, C, KD, LDK, THREADS>(s_k, pk + u0 * dir * a.k.st, dir * a.k.st, a.kd, n, vec_k);
    stage<T, C, NV, LDV, THREADS>(s_v, pv + u0 * dir * a.v.st, dir * a.v.st, vw, n, vec_v);
    if constexpr (kDecay) stage<T, C, NV, LDV, THREADS>(s_dy, pdy + u0 * a.dy.st, a.dy.st, vw, n, vec_dy);
    __syncthreads();

    if constexpr (kOut) {
      // P = W o Q K^T, tile (it, jt) at a time, transposed so that a lane holds 4 steps j of a row i
      for (int tile = wave; tile < IT * (IT + 1) / 2; tile += NW) {
        int it = 0, jt = tile;
        while (jt > it) jt -= ++it;
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < KD; kk += CK)
          acc = M::mma(M::row(s_k, LDK, 16 * jt, kk, lane), M::row(s_q, LDK, 16 * it, kk, lane), acc);
        const int i = 16 * it + m;
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * jt + q4 + r;
          const bool kept = j <= i && (B == 0 || seen(i) == seen(j));
          float w = s_pw[kept ? i - j : 0] * a.scale_p;
          if (kDecay) w *= (float)(i - j);
          p[r] = kept ? acc[r] * w : 0.0f;
        }
        T* dst = s_p + i * LDP + 16 * jt + q4;
        if constexpr (sizeof(T) == 2) {
          if constexpr (kDecay) {
            float lo[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float hi = cut16(p[r]);
              lo[r] = p[r] - hi;
              p[r] = hi;
            }
            *reinterpret_cast<uint2*>(s_p2 + i * LDP + 16 * jt + q4) =
                make_uint2(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]));
          }
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
        } else {
          *reinterpret_cast<f32x4*>(dst) = f32x4{p[0], p[1], p[2], p[3]};
        }
      }
      __syncthreads();
    }

    // this wave's columns of V, contracted over the steps
    Frag vf[C / CK];
    float x[C / CK][E], x2[kDecay ? C / CK : 1][E];
    float odd = 0.0f;  // NaN if any of the values is not finite
    const int total = seen(n - 1);
#pragma unroll
    for (int s = 0; s < C / CK; ++s) {
      vf[s] = M::col(s_v, LDV, CK * s, 16 * wave, lane);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int j = CK * s + E * (lane >> 4) + e;
        const int left = n - 1 - j;
        const float v = M::at(vf[s], e) * (s_pw[left < 0 ? 0 : left + sh] * a.scale_upd);
        odd = __builtin_fmaf(v, 0.0f, odd);
        const bool kept = left >= 0 && (B == 0 || seen(j) == total);
        x[s][e] = kept ? v : 0.0f;
        if constexpr (kDecay) x2[s][e] = kept ? v * (float)left : 0.0f;
      }
    }
    // Values that are not finite are left out of the product with P, whose zeros
    // above the diagonal they would turn into NaN, and added apart.
    const bool careful = __any(!(odd == 0.0f));
    if (careful) {
#pragma unroll
      for (int s = 0; s < C / CK; ++s)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!finite_f32(M::at(vf[s], e))) M::zero(vf[s], e);
    }

    if constexpr (kOut) {
      f32x4 acc[IT], acc_r[kDecay ? IT : 1];
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        acc[it] = f32x4{0, 0, 0, 0};
        if constexpr (kDecay) acc_r[it] = f32x4{0, 0, 0, 0};
      }
      // (Q S)^T: a lane holds 4 value columns of a step
#pragma unroll
      for (int kk = 0; kk < KD / CK; ++kk) {
        float sv[E], rv[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          sv[e] = S[kk * (CK / 16) + e / 4][e % 4];
          if constexpr (kDecay) rv[e] = R[kk * (CK / 16) + e / 4][e % 4];
        }
        const auto ps = parts_of<NS>(sv);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const Frag fq = M::row_as_state(s_q, LDK, 16 * it, kk * CK, lane);
#pragma unroll
          for (int k = 0; k < NS; ++k) acc[it] = M::mma(ps.f[k], fq, acc[it]);
          if constexpr (kDecay) {
            const auto pr = parts_of<NS>(rv);
#pragma unroll
            for (int k = 0; k < NS; ++k) acc_r[it] = M::mma(pr.f[k], fq, acc_r[it]);
          }
        }
      }
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const int i = 16 * it + m;
        const bool kept = B == 0 || seen(i) == 0;
        const float w = s_pw[i + 1 - sh] * a.scale_in;
        f32x4 o;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          o[r] = acc[it][r];
          if constexpr (kDecay) o[r] = __builtin_fmaf(o[r], (float)(i + 1), acc_r[it][r]);
          o[r] = kept ? o[r] * w : 0.0f;
        }
#pragma unroll
        for (int s = 0; s < C / CK; ++s) {
          if (CK * s >= 16 * (it + 1)) continue;
          o = M::mma(vf[s], M::row(s_p, LDP, 16 * it, CK * s, lane), o);
          if constexpr (kDecay && sizeof(T) == 2) o = M::mma(vf[s], M::row(s_p2, LDP, 16 * it, CK * s, lane), o);
        }
        if (careful) {  // the values left out of vf, to the steps that take them
          for (int j = 0; j <= min(i, n - 1); ++j) {
            if (B != 0 && seen(j) != seen(i)) continue;
            const float p = Elem<T>::load(s_p + i * LDP + j);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float v = Elem<T>::load(s_v + j * LDV + 16 * wave + q4 + r);
              if (!finite_f32(v)) o[r] = __builtin_fmaf(p, v, o[r]);
            }
          }
        }
        acc[it] = o;
      }
      if constexpr (kDecay) {
        float sum = 0.0f;
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = 16 * it + m, c = 16 * wave + q4 + r;
            if (i < n && c < vw)
              sum = __builtin_fmaf(acc[it][r], Elem<T>::load(s_dy + i * LDV + c), sum);
          }
        dg += (double)sum;
      } else {
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const int i = 16 * it + m, u = u0 + i;
          if (u < u_end) {
            const int t = u < len && a.rev ? len - 1 - u : u;
            const int64_t at = (((int64_t)b * L + t) * a.heads + h) * a.vd + v0 + 16 * wave + q4;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float v = i < n ? acc[it][r] : 0.0f;
              if (16 * wave + q4 + r < vw) {
                if (a.out_f32) static_cast<float*>(a.out)[at + r] = v;
                else Elem<T>::store(out + at + r, v);
              }
            }
          }
        }
      }
    }

    // the state behind the chunk
    const float pass = s_pw[n];
    if (MODE == kAttnSegments) cut |= B != 0;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (kDecay) R[t][r] = total == 0 ? __builtin_fmaf(S[t][r], (float)n, R[t][r]) * pass : 0.0f;
        S[t][r] = total == 0 ? S[t][r] * pass : 0.0f;
      }
#pragma unroll
    for (int s = 0; s < C / CK; ++s) {
      const auto px = parts_of<NU>(x[s]);
      const auto px2 = parts_of<NU>(x2[kDecay ? s : 0]);
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        Frag kf = M::col(s_k, LDK, CK * s, 16 * t, lane);
        if (B != 0) {  // not even a NaN of the steps before the last start
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (seen(CK * s + E * (lane >> 4) + e) != total) M::zero(kf, e);
        }
#pragma unroll
        for (int k = 0; k < NU; ++k) S[t] = M::mma(kf, px.f[k], S[t]);
        if constexpr (kDecay) {
#pragma unroll
          for (int k = 0; k < NU; ++k) R[t] = M::mma(kf, px2.f[k], R[t]);
        }
      }
    }
  }

  const int64_t mat = (int64_t)a.kd * a.vd;
  if constexpr (MODE == kAttnSegments) {
    const int steps = min(max(len - u_begin, 0), u_end - u_begin);
    through = cut ? 0.0f : decay_pow(g, (float)steps);
    if (vb == 0 && threadIdx.x == 0) a.seg_through[head * a.nseg + seg] = through;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * t + q4 + r;
        if (row < a.kd && col < a.vd)
          a.seg_state[(head * a.nseg + seg + 1) * mat + (int64_t)row * a.vd + col] = S[t][r];
      }
  } else if constexpr (MODE == kAttnOut) {
    if (a.state_out != nullptr && seg == a.nseg - 1) {
      // backward in time nothing passes a first step that starts a sequence
      const bool gone = a.rev && a.starts != nullptr && len > 0 && a.starts[(int64_t)b * L] != 0;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * t + q4 + r;
          if (row < a.kd && col < a.vd)
            a.state_out[head * mat + (a.transposed ? (int64_t)col * a.kd + row : (int64_t)row * a.vd + col)] =
                gone ? 0.0f : S[t][r];
        }
    }
  } else {
    if (dlast != nullptr) {
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * t + q4 + r;
          if (row < a.kd && col < a.vd) sum = __builtin_fmaf(R[t][r], dlast[head * mat + (int64_t)row * a.vd + col], sum);
        }
      dg += (double)sum;
    }
    dg = wave_sum(dg);
    if (lane == 0) s_sum[wave] = dg;
    __syncthreads();
    if (threadIdx.x == 0) {
      double sum = 0.0;
      for (int w = 0; w < NW; ++w) sum += s_sum[w];
      a.part[((int64_t)h * a.batch + b) * nvb + vb] = sum;
    }
  }
}

// The states entering the segments from what each adds: S <- through S + added, a
// thread an element.
__global__ __launch_bounds__(256) void attn_carry_kernel(float* __restrict__ state, const float* __restrict__ through,
                                                         const float* __restrict__ state_in, int kd, int vd, int nseg,
                                                         int transposed, int64_t n) {
  const int64_t i = group_index() * 256 + threadIdx.x;
  if (i >= n) return;
  const int mat = kd * vd;
  const int64_t head = i / mat;
  const int e = (int)(i - head * mat), row = e / vd, col = e - row * vd;
  float s = 0.0f;
  if (state_in != nullptr) s = state_in[head * mat + (transposed ? col * kd + row : e)];
  float* p = state + head * nseg * mat + e;
  const float* th = through + head * nseg;
  for (int k = 0; k + 1 < nseg; ++k) {
    const float added = p[(int64_t)(k + 1) * mat];
    s = th[k] == 0.0f ? added : __builtin_fmaf(th[k], s, added);
    p[(int64_t)(k + 1) * mat] = s;
  }
}

// Sums over the heads that share one, in their order.
template <typename T>
__global__ __launch_bounds__(256) void attn_gather_kernel(const float* __restrict__ part, T* __restrict__ out, int heads,
                                                          int n, int width, int64_t total) {
  const int64_t i = group_index() * 256 + threadIdx.x;
  if (i >= total) return;
  const int per = heads / n;
  const int64_t row = i / width;  // (batch, step, shared head)
  const int c = (int)(i - row * width);
  const float* p = part + row * per * width + c;
  float s = 0.0f;
  for (int k = 0; k < per; ++k) s += p[(int64_t)k * width];
  Elem<T>::store(out + i, s);
}

__global__ __launch_bounds__(64) void attn_decay_sum_kernel(const double* __restrict__ part, float* __restrict__ out,
                                                            int per) {
  const double* p = part + (int64_t)blockIdx.x * per;
  double s = 0.0;
  for (int i = threadIdx.x; i < per; i += 64) s += p[i];
  s = wave_sum(s);
  if (threadIdx.x == 0) out[blockIdx.x] = (float)s;
}

// One token: S <- e^g S + k v^T, y = scale q S.  A workgroup takes a (batch row,
// head) and 64 value columns, a lane one of them, a wave every fourth row.
template <typename T>
__global__ __launch_bounds__(256) void attn_step_kernel(const AttnStep a) {
  __shared__ float s_y[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int nvb = (a.vd + 63) / 64;
  int64_t id = group_index();
  if (id >= (int64_t)a.batch * a.heads * nvb) return;
  const int vb = (int)(id % nvb);
  id /= nvb;
  const int h = (int)(id % a.heads), b = (int)(id / a.heads);
  const int col = vb * 64 + lane;
  const auto base = [&](const AttnView& w) { return static_cast<const T*>(w.p) + b * w.sb + (h / w.share) * w.sh; };
  const T *pq = base(a.q), *pk = base(a.k), *pv = base(a.v);
  const bool first = a.starts != nullptr && a.starts[b] != 0;
  const float decay = decay_pow(a.g[h], 1.0f);
  const int64_t at = ((int64_t)b * a.heads + h) * a.kd * a.vd;
  float y = 0.0f;
  if (col < a.vd) {
    const float v = Elem<T>::load(pv + col);
    for (int row = wave; row < a.kd; row += 4) {
      const int64_t e = at + (int64_t)row * a.vd + col;
      const float kv = Elem<T>::load(pk + row) * v;
      const float s = first ? kv : __builtin_fmaf(decay, a.state[e], kv);
      a.state_out[e] = s;
      y = __builtin_fmaf(Elem<T>::load(pq + row), s, y);
    }
  }
  s_y[wave][lane] = y;
  __syncthreads();
  if (wave == 0 && col < a.vd) {
    y = ((s_y[0][lane] + s_y[1][lane]) + (s_y[2][lane] + s_y[3][lane])) * a.scale;
    Elem<T>::store(static_cast<T*>(a.y) + ((int64_t)b * a.heads + h) * a.vd + col, y);
  }
}

namespace {

constexpr int kColumns = 128;  // value columns of a workgroup of 8 waves

template <typename T, int KD, int NW, int MODE>
hipError_t sweep(const AttnSweep& a, const float* dlast, hipStream_t stream) {
  const int nvb = (a.vd + 16 * NW - 1) / (16 * NW);
  const int nsegs = MODE == kAttnSegments ? a.nseg - 1 : MODE == kAttnDecay ? 1 : a.nseg;
  attn_sweep_kernel<T, KD, NW, MODE>
      <<<grid_of((int64_t)a.batch * a.heads * nvb * nsegs, 64 * NW), 64 * NW, 0, stream>>>(a, dlast);
  return hipGetLastError();
}

template <typename T, int MODE>
hipError_t sweep_of(const AttnSweep& a, const float* dlast, hipStream_t stream) {
  const int kd = a.kd <= 64 ? 64 : a.kd <= 128 ? 128 : 256;
  if (a.vd <= 64) {
    if (kd == 64) return sweep<T, 64, 4, MODE>(a, dlast, stream);
    if (kd == 128) return sweep<T, 128, 4, MODE>(a, dlast, stream);
    return sweep<T, 256, 4, MODE>(a, dlast, stream);
  }
  if (kd == 64) return sweep<T, 64, 8, MODE>(a, dlast, stream);
  if (kd == 128) return sweep<T, 128, 8, MODE>(a, dlast, stream);
  return sweep<T, 256, 8, MODE>(a, dlast, stream);
}

template <typename T>
hipError_t run_sweep(const AttnSweep& a, hipStream_t stream) {
  if (a.nseg > 1) {
    hipError_t e = sweep_of<T, kAttnSegments>(a, nullptr, stream);
    if (e != hipSuccess) return e;
    const int64_t n = (int64_t)a.batch * a.heads * a.kd * a.vd;
    attn_carry_kernel<<<grid_of((n + 255) / 256, 256), 256, 0, stream>>>(a.seg_state, a.seg_through, a.state_in, a.kd,
                                                                         a.vd, a.nseg, a.transposed, n);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return sweep_of<T, kAttnOut>(a, nullptr, stream);
}

}  // namespace

int attn_column_blocks(int vd) { return vd <= 64 ? 1 : (vd + kColumns - 1) / kColumns; }

AttnSplit attn_split(int batch, int heads, int64_t seqlen, int vd) {
  // two workgroups for each of the 256 CUs, segments of 4 chunks at least
  const int64_t groups = (int64_t)batch * heads * attn_column_blocks(vd);
  const int64_t chunks = (seqlen + kAttnChunk - 1) / kAttnChunk;
  int64_t want = groups >= 512 || groups == 0 ? 1 : 512 / groups;
  if (want > chunks / 4) want = chunks / 4;
  if (want < 2) return AttnSplit{1, (chunks > 0 ? chunks : 1) * kAttnChunk};
  const int64_t per = (chunks + want - 1) / want;
  return AttnSplit{(int)((chunks + per - 1) / per), per * kAttnChunk};
}

hipError_t launch_attn_sweep(const AttnSweep& a, hipStream_t stream) {
  return a.dtype == Dtype::BF16 ? run_sweep<uint16_t>(a, stream) : run_sweep<float>(a, stream);
}

hipError_t launch_attn_decay_grad(const AttnSweep& a, const float* dlast, float* dlog_decay, hipStream_t stream) {
  const hipError_t e = a.dtype == Dtype::BF16 ? sweep_of<uint16_t, kAttnDecay>(a, dlast, stream)
                                              : sweep_of<float, kAttnDecay>(a, dlast, stream);
  if (e != hipSuccess) return e;
  attn_decay_sum_kernel<<<a.heads, 64, 0, stream>>>(a.part, dlog_decay, a.batch * attn_column_blocks(a.vd));
  return hipGetLastError();
}

hipError_t launch_attn_gather(const float* part, void* out, int64_t rows, int heads, int n, int width, Dtype dtype,
                              hipStream_t stream) {
  const int64_t total = rows * n * width;
  const dim3 grid = grid_of((total + 255) / 256, 256);
  if (dtype == Dtype::BF16)
    attn_gather_kernel<uint16_t><<<grid, 256, 0, stream>>>(part, static_cast<uint16_t*>(out), heads, n, width, total);
  else
    attn_gather_kernel<float><<<grid, 256, 0, stream>>>(part, static_cast<float*>(out), heads, n, width, total);
  return hipGetLastError();
}

hipError_t launch_attn_step(const AttnStep& a, hipStream_t stream) {
  const int nvb = (a.vd + 63) / 64;
  const dim3 grid = grid_of((int64_t)a.batch * a.heads * nvb, 256);
  if (a.dtype == Dtype::BF16) attn_step_kernel<uint16_t><<<grid, 256, 0, stream>>>(a);
  else attn_step_kernel<float><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace ssm
