// gated.hip -- the gated linear recurrence over whole sequences, its backward
// pass and its one-token step, for gfx950 (include/ssm_gated.h states it).
//
// Per channel h_t = a_t h_{t-1} + v_t with a_t = exp(A g_t), v_t = w_t u_t.
// There is one state per channel, so nothing is gained by giving a lane a
// channel as the selective scan does: a wave walks one row (b, d) in blocks of
// 512 steps, each lane holding 8 consecutive ones (16 bytes of bf16), so every
// access of a wave is 1 KiB in one piece.  A lane composes its 8 steps into
// the map h -> P h + Q, the maps are composed over the wave by a prefix (six
// DPP rounds), and each lane reruns its steps from the state entering them:
// one pass over HBM.  P = exp2 of the sum of the steps' exponents.
//
// Rows of at most 256 steps (W = 0) share a wave: a power of two of lanes to each,
// whose first applies its map to the row's entering state and from then on
// forgets what is before it, as at a start.
//
// Where there are too few rows to fill the chip with a wave each, W waves take a
// row's blocks in turn, W at a time: each wave's map over its block goes to the
// others through LDS (a barrier for every W blocks), and each applies those before
// its own to the row's state.
//
// The backward pass walks the blocks from last to first.  It forms the gates
// again, the states from the block's kept entering state, and the adjoint
// lambda_t = dh_t + a_{t+1} lambda_{t+1} by the same prefix over the mirrored
// lanes (its map m -> P m + Q carries m_t = a_t lambda_t to the left).
#include "gated_math.hpp"
#include "row_slices.hpp"
#include "ssm_kernels.hpp"

namespace ssm {

namespace {

// Waves of a workgroup with W waves to a row: 4 of one row or several each, else
// those of one row.
constexpr int group_waves(int W) { return W <= 1 ? 4 : W; }

struct GatedSizes {
  int rows, dim;
  int seqlen, nblk;
  int lanes;  // lanes of a row (W = 0; else 64)
  int once;   // inputs are read past the caches
};

// Where the calling lane works.  row is the wave's own but for W = 0.
template <int W>
struct Place {
  int row;
  int lane, w0;     // lane among the row's lanes; wave among the row's waves
  bool live, last;  // a row of the call; the row's last lane
};

template <int W>
__device__ __forceinline__ Place<W> place_of(const GatedSizes& p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Place<W> q;
  if constexpr (W == 0) {
    q.lane = lane & (p.lanes - 1);
    const int64_t row = group_index() * (group_waves(W) * 64 / p.lanes) + threadIdx.x / p.lanes;
    q.live = row < p.rows;
    q.row = q.live ? (int)row : 0;
    q.w0 = 0;
    q.last = q.lane == p.lanes - 1;
  } else {
    q.lane = lane;
    const int64_t row = W == 1 ? group_index() * group_waves(W) + wave : blockIdx.x;
    q.live = row < p.rows;  // (with more waves to a row the grid is the rows)
    q.row = (int)row;
    q.w0 = W == 1 ? 0 : wave;
    q.last = lane == 63;
  }
  return q;
}

// The steps that a lane holds of its wave's block: kRun in a row for bf16, one
// access of 16 bytes.  For float32 that would be two accesses with gaps of 16
// bytes between the lanes; the block is taken as two halves instead, 4 steps of
// each to a lane, so that every access of a wave is 1 KiB in one piece, and the
// prefix runs once for each half (backward of batch 8, dim 1536, L 2047: 163 us with
// gaps, 156; forward of L 2048: 104, 94).  Rows that share a wave keep kRun in a
// row.
template <typename T, int W>
struct Steps {
  static constexpr int NH = sizeof(T) == 4 && W > 0 ? 2 : 1;
  static constexpr int RN = kRun / NH;          // steps of a run
  static constexpr int kGap = kGatedBlock / NH;  // from a lane's run to its next

  // steps 0 .. RN-1 at p and (halves) at p + kGap, `left` steps from p to the row's end
  template <bool ONCE>
  __device__ __forceinline__ static RunWords<T> load(const T* p, int64_t left) {
    if constexpr (NH == 1) {
      return load_run<T, ONCE>(p, clamped(left));
    } else {
      RunWords<T> r;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const T* q = p + h * kGap;
        const int valid = clamped(left - h * kGap);
        if (valid >= RN) {
          const auto* at = reinterpret_cast<const typename RunWords<T>::vec4*>(q);
          const auto v = ONCE ? __builtin_nontemporal_load(at) : *at;
          r.w[4 * h] = v.x; r.w[4 * h + 1] = v.y; r.w[4 * h + 2] = v.z; r.w[4 * h + 3] = v.w;
        } else {
#pragma unroll
          for (int k = 0; k < RN; ++k) r.w[4 * h + k] = k < valid ? __float_as_uint(q[k]) : 0u;
        }
      }
      return r;
    }
  }
  __device__ __forceinline__ static void store(T* p, int64_t left, const float (&f)[kRun]) {
    if constexpr (NH == 1) {
      store_run<T, sizeof(T) == 2>(p, clamped(left), f);
    } else {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        T* q = p + h * kGap;
        const int valid = clamped(left - h * kGap);
        if (valid >= RN) {
          typename RunWords<T>::vec4 v;
          v.x = __float_as_uint(f[4 * h]); v.y = __float_as_uint(f[4 * h + 1]);
          v.z = __float_as_uint(f[4 * h + 2]); v.w = __float_as_uint(f[4 * h + 3]);
          __builtin_nontemporal_store(v, reinterpret_cast<typename RunWords<T>::vec4*>(q));
        } else {
#pragma unroll
          for (int k = 0; k < RN; ++k)
            if (k < valid) q[k] = f[4 * h + k];
        }
      }
    }
  }
  // bit k: a sequence starts at the lane's step k
  __device__ __forceinline__ static uint32_t starts(const uint8_t* p, int64_t left) {
    if constexpr (NH == 1) {
      return load_starts<kRun>(p, clamped(left));
    } else {
      return load_starts<RN>(p, clamped(left)) | load_starts<RN>(p + kGap, clamped(left - kGap)) << RN;
    }
  }
  // bit k: the lane's step k is in the row
  __device__ __forceinline__ static uint32_t inside(int64_t left) {
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < NH; ++h) m |= ((1u << clamped(left - h * kGap)) - 1u) << (h * RN);
    return m;
  }
  __device__ __forceinline__ static int clamped(int64_t left) { return left >= RN ? RN : left < 0 ? 0 : (int)left; }
};

// A wave's total map, for the other waves of its row; two buffers, so that one
// barrier for every W blocks is enough.
template <int W>
struct RowMaps {
  float P[2][W > 0 ? W : 1], Q[2][W > 0 ? W : 1];
};

// The value that enters wave `w` of a row's W, whose waves map it in the order
// 0, 1, .. (the forward) or W-1, W-2, .. (the backward): `in` mapped by those
// before it.  `in` becomes the value after all of them.
template <bool CUT, int W, bool REVERSE>
__device__ __forceinline__ float through_waves(RowMaps<W>& s, int turn, int w, float P, float Q, float& in) {
  if constexpr (W <= 1) {
    return in;
  } else {
    // lane 63 of the prefix holds the wave's total
    if ((threadIdx.x & 63) == 63) {
      s.P[turn][w] = P;
      s.Q[turn][w] = Q;
    }
    __syncthreads();
    float mine = in;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const int k = REVERSE ? W - 1 - j : j;
      if (k == w) mine = in;
      in = apply_map<CUT>(s.P[turn][k], s.Q[turn][k], in);
    }
    return mine;
  }
}

// Where A > 0 the decays grow: over several runs they may multiply past float32
// while every state is inside it (0 until late, or small), and a composed map would
// form inf * 0.  A wave with a channel whose decays might pass 2^100 over a block
// (what is left of the exponents is for the inputs) composes nothing: it takes a step
// a lane and goes from lane to lane, and the row's other waves have nothing to do
// (batch 8, dim 5120, L 2048 bf16 without gates, no channel so, one in 100, all:
// forward 91, 168, 890 us, backward 180, 320, 1950).
//
// The largest A log2(e) g of a step that is safe, over a block:
constexpr float kSafeGrowth = 100.0f / kGatedBlock;

// Whether a channel of the wave may pass it (A2 = A log2 e), as far as A says.
template <int RULE>
__device__ __forceinline__ bool grows_fast(float A2) {
  return __any(A2 > ((RULE & kGateSoftplus) != 0 ? 0.0f : kSafeGrowth));
}

// Whether one does, anywhere in its row: a sigmoid is at most 1, for a softplus the
// row's waves look for the largest r.
template <typename T, int RULE, int W>
__device__ __forceinline__ bool may_overflow(const T* r, float A2, float rb, const Place<W>& at, const GatedSizes& p,
                                             float (&s_most)[W > 1 ? W : 1]) {
  float g = 1.0f;
  if constexpr ((RULE & kGateSoftplus) != 0) {
    float most = -__builtin_inff();
    const int lanes = W == 0 ? p.lanes : 64;
#pragma unroll 1
    for (int64_t t = ((int64_t)at.w0 * lanes + at.lane) * kRun; t < p.seqlen; t += (W > 1 ? W : 1) * lanes * kRun) {
      const int64_t left = p.seqlen - t;
      float f[kRun];
      run_floats<T>(load_run(r + t, left < kRun ? (int)left : kRun), f);
#pragma unroll
      for (int k = 0; k < kRun; ++k) most = k < left ? __builtin_fmaxf(most, f[k]) : most;
    }
    for (int off = 1; off < lanes; off <<= 1) most = __builtin_fmaxf(most, __shfl_xor(most, off));
    if constexpr (W > 1) {
      if (at.lane == 0) s_most[at.w0] = most;
      __syncthreads();
      for (int w = 0; w < W; ++w) most = __builtin_fmaxf(most, s_most[w]);
    }
    g = softplus_f32(most + rb);
  }
  return __any(A2 * g > kSafeGrowth);
}

// What enters each lane's step: `first` for the row's first lane (as `next` hands
// it), for the others what `step` makes of the lane before's, known after as many
// turns as there are lanes before.
template <typename S, typename N>
__device__ __forceinline__ float lanes_in_turn(int lanes, float first, S&& step, N&& next) {
  float in = first;
#pragma unroll 1
  for (int n = 1; n < lanes; ++n) in = next(step(in));
  return in;
}

}  // namespace

// g of a step from its raw r: nb = -r_bias log2(e).
template <int RULE>
__device__ __forceinline__ float gate_value(float r, float rb, float nb) {
  if constexpr ((RULE & kGateSoftplus) != 0) return softplus_f32(r + rb);
  else return sigmoid_f32(r, nb);
}

template <typename T, int RULE, bool IG, bool ZG, int W>
__global__ __launch_bounds__(64 * group_waves(W)) void gated_fwd_kernel(
    const T* __restrict__ x, const T* __restrict__ r, const float* __restrict__ A,
    const float* __restrict__ r_bias, const T* __restrict__ ig, const float* __restrict__ i_bias,
    const T* __restrict__ z, const uint8_t* __restrict__ starts, const float* __restrict__ h0,
    T* __restrict__ y, float* __restrict__ last_state, float* __restrict__ ckpt, const GatedSizes p) {
  using ST = Steps<T, W>;
  constexpr int NH = ST::NH, RN = ST::RN;
  [[maybe_unused]] __shared__ RowMaps<W> maps;
  [[maybe_unused]] __shared__ float s_most[W > 1 ? W : 1];
  const Place<W> at = place_of<W>(p);
  if (W > 0 && !at.live) return;
  const int lane = at.lane, row = at.row, w0 = at.w0;
  const int b = row / p.dim, d = row - b * p.dim;
  const float A2 = A[d] * kLog2e;
  const float rb = r_bias != nullptr ? r_bias[d] : 0.0f, nrb = -rb * kLog2e;
  const float nib = IG && i_bias != nullptr ? -i_bias[d] * kLog2e : 0.0f;
  const int64_t base = (int64_t)row * p.seqlen;
  float H = h0 != nullptr ? h0[row] : 0.0f;

  // the row's steps in turn
  auto in_turn = [&] {
    const int lanes = W == 0 ? p.lanes : 64, place = threadIdx.x & 63;
#pragma unroll 1
    for (int c = 0; c < p.seqlen; c += lanes) {
      const int t = c + lane;
      const bool in = at.live && t < p.seqlen;
      float a = 1.0f, q = 0.0f;
      if (in) {
        const Gate g = gate_of<RULE>(gate_value<RULE>(Elem<T>::load(r + base + t), rb, nrb), A2);
        a = starts != nullptr && starts[(int64_t)b * p.seqlen + t] != 0 ? 0.0f : g.a;
        q = g.w * Elem<T>::load(x + base + t);
        if constexpr (IG) q *= sigmoid_f32(Elem<T>::load(ig + base + t), nib);
      }
      auto step = [&](float v) { return apply_map<true>(a, q, v); };
      const float from = lanes_in_turn(lanes, H, step, [&](float v) {
        const float before = lane_before(v, H);
        return lane == 0 ? H : before;
      });
      const float h = step(from);
      if (in) {
        if (ckpt != nullptr && t % kGatedBlock == 0) ckpt[((int64_t)b * p.nblk + t / kGatedBlock) * p.dim + d] = from;
        float o = h;
        if constexpr (ZG) o *= silu_f32(Elem<T>::load(z + base + t));
        Elem<T>::store(y + base + t, o);
      }
      H = __shfl(h, place | (lanes - 1));
    }
  };

  // whether the row cannot be composed
  auto must_turn = [&] {
    return grows_fast<RULE>(A2) && may_overflow<T, RULE, W>(r + base, A2, rb, at, p, s_most);
  };

  // one block a wave; WHOLE: every step of the W blocks is in the row; ONCE:
  // inputs read past the caches
  auto blocks = [&](int b0, int turn, auto whole, auto once) {
    constexpr bool WHOLE = decltype(whole)::value, ONCE = decltype(once)::value;
    const int blk = b0 + w0;  // past the last block: no steps, the identity
    const int64_t t0 = (int64_t)blk * kGatedBlock + lane * RN;
    const int64_t left = WHOLE ? kGatedBlock : at.live ? p.seqlen - t0 : 0;
    RunWords<T> wr, wx, wi, wz;
    auto load = [&] {
      wr = ST::template load<ONCE>(r + base + t0, left);
      wx = ST::template load<ONCE>(x + base + t0, left);
      if constexpr (IG) wi = ST::template load<ONCE>(ig + base + t0, left);
      if constexpr (ZG) wz = ST::template load<ONCE>(z + base + t0, left);
    };
    load();
    if constexpr (W == 0) {
      // Asked with the rows' only loads on their way, which would else wait for A (batch
      // 64, dim 1536, L 200 float32: 72 us, 80); they are not held meanwhile.
      if (grows_fast<RULE>(A2)) {
        if (must_turn()) return in_turn();
        asm volatile("" ::: "memory");
        load();
      }
    }
    uint32_t cut = 0;
    if (starts != nullptr) cut = ST::starts(starts + (int64_t)b * p.seqlen + t0, left);
    const uint32_t in = WHOLE ? ~0u : ST::inside(left);

    float fr[kRun], fx[kRun], fi[kRun], a[kRun], q[kRun];
    run_floats<T>(wr, fr);
    run_floats<T>(wx, fx);
    if constexpr (IG) run_floats<T>(wi, fi);
    float S[NH];  // exponent of a run's decay
#pragma unroll
    for (int h = 0; h < NH; ++h) S[h] = 0.0f;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const Gate g = gate_of<RULE>(gate_value<RULE>(fr[k], rb, nrb), A2);
      a[k] = g.a;
      q[k] = g.w * fx[k];
      if constexpr (IG) q[k] *= sigmoid_f32(fi[k], nib);
      if (!WHOLE && !(in & (1u << k))) {
        a[k] = 1.0f;
        q[k] = 0.0f;
      } else {
        S[k / RN] += g.e2;
      }
    }
    float h_in;
    auto rerun = [&](auto cuts) {
      constexpr bool CUT = decltype(cuts)::value;
      float P[NH], Q[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        P[h] = __builtin_fmaxf(exp2_hw(S[h]), kMinNormal);
        Q[h] = 0.0f;
#pragma unroll
        for (int k = h * RN; k < (h + 1) * RN; ++k) {
          if (CUT && (cut & (1u << k))) a[k] = 0.0f;
          Q[h] = apply_map<CUT>(a[k], q[k], Q[h]);
        }
        if (CUT && (cut >> (h * RN) & ((1u << RN) - 1u)) != 0) P[h] = 0.0f;
        if (W == 0 && lane == 0) {
          Q[h] = apply_map<true>(P[h], Q[h], H);
          P[h] = 0.0f;
        }
        wave_prefix<CUT>(P[h], Q[h]);
      }
      float Pt = P[0], Qt = Q[0];
      if constexpr (NH == 2) {
        Pt = P[1], Qt = Q[1];
        compose_map<CUT>(Pt, Qt, P[0], Q[0]);
      }
      h_in = through_waves<CUT, W, false>(maps, turn, w0, Pt, Qt, H);
      float from = h_in;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float end = apply_map<CUT>(P[h], Q[h], from);
        float v = lane_before(end, from);
        if (W == 0 && lane == 0) v = H;
        if constexpr (W == 0) H = end;
        else from = lane_value(end, 63);
#pragma unroll
        for (int k = h * RN; k < (h + 1) * RN; ++k) q[k] = v = apply_map<CUT>(a[k], q[k], v);
      }
      if constexpr (W == 1) H = from;
    };
    if (W == 0 || starts != nullptr) rerun(BoolC<true>{});
    else rerun(BoolC<false>{});
    if (ckpt != nullptr && lane == 0 && at.live && blk < p.nblk)
      ckpt[((int64_t)b * p.nblk + blk) * p.dim + d] = h_in;
    if constexpr (ZG) {
      float fz[kRun];
      run_floats<T>(wz, fz);
#pragma unroll
      for (int k = 0; k < kRun; ++k) q[k] *= silu_f32(fz[k]);
    }
    ST::store(y + base + t0, left, q);
  };
  if constexpr (W == 0) {
    blocks(0, 0, BoolC<false>{}, BoolC<false>{});
  } else if (must_turn()) {
    if (w0 == 0) in_turn();
  } else {
    int b0 = 0, turn = 0;
    auto wholes = [&](auto once) {
      for (; (int64_t)(b0 + W) * kGatedBlock <= p.seqlen; b0 += W, turn ^= 1) blocks(b0, turn, BoolC<true>{}, once);
    };
    if (p.once) wholes(BoolC<true>{});
    wholes(BoolC<false>{});
    if (b0 < p.nblk) blocks(b0, turn, BoolC<false>{}, BoolC<false>{});
  }
  if (last_state != nullptr && at.live && at.last && w0 == 0) last_state[row] = H;
}

template <typename T, int RULE, bool IG, bool ZG, int W>
__global__ __launch_bounds__(64 * group_waves(W)) void gated_bwd_kernel(
    const T* __restrict__ x, const T* __restrict__ r, const float* __restrict__ A,
    const float* __restrict__ r_bias, const T* __restrict__ ig, const float* __restrict__ i_bias,
    const T* __restrict__ z, const uint8_t* __restrict__ starts, const float* __restrict__ ckpt,
    const T* __restrict__ dy, const float* __restrict__ dlast, T* __restrict__ dx, T* __restrict__ dr,
    T* __restrict__ di, T* __restrict__ dz, float* __restrict__ row_dA, float* __restrict__ row_drb,
    float* __restrict__ row_dib, float* __restrict__ dh0, const GatedSizes p) {
  using ST = Steps<T, W>;
  constexpr int NH = ST::NH, RN = ST::RN;
  [[maybe_unused]] __shared__ RowMaps<W> maps;
  [[maybe_unused]] __shared__ float s_most[W > 1 ? W : 1];
  const Place<W> at = place_of<W>(p);
  if (W > 0 && !at.live) return;
  const int lane = at.lane, row = at.row, w0 = at.w0;
  const int b = row / p.dim, d = row - b * p.dim;
  const float Ad = A[d], A2 = Ad * kLog2e;
  const float rb = r_bias != nullptr ? r_bias[d] : 0.0f, nrb = -rb * kLog2e;
  const float nib = IG && i_bias != nullptr ? -i_bias[d] * kLog2e : 0.0f;
  const int64_t base = (int64_t)row * p.seqlen;
  float M = dlast != nullptr ? dlast[row] : 0.0f;  // a_{t+1} lambda_{t+1} entering from the right
  // the row's sums, over up to 2^31 steps: in float64 across blocks
  double sA = 0.0, srb = 0.0, sib = 0.0;

  // the row's steps in turn, a block's states first (those that enter its 8 pieces
  // and less are kept, each lane its own copy)
  __shared__ float s_enter[W == 1 || W == 0 ? group_waves(W) : 1][8][64];
  auto in_turn = [&] {
    const int lanes = W == 0 ? p.lanes : 64, place = threadIdx.x & 63;
    float(*const enter)[64] = s_enter[W <= 1 ? threadIdx.x >> 6 : 0];
#pragma unroll 1
    for (int blk = p.nblk - 1; blk >= 0; --blk) {
      const int t0 = blk * kGatedBlock;
      const int steps = p.seqlen - t0 < kGatedBlock ? p.seqlen - t0 : kGatedBlock;
      const int pieces = (steps + lanes - 1) / lanes;
      float from = ckpt[((int64_t)b * p.nblk + blk) * p.dim + d];
#pragma unroll 1
      for (int n = 0; n < 2 * pieces - 1; ++n) {
        const bool ahead = n < pieces - 1;  // only the states
        const int c = ahead ? n : 2 * pieces - 2 - n;
        const int t = t0 + c * lanes + lane;
        const bool in = at.live && t < p.seqlen;
        const bool cut = in && starts != nullptr && starts[(int64_t)b * p.seqlen + t] != 0;
        float v = 0.0f, slope = 0.0f, u = 0.0f, xv = 0.0f, s_i = 1.0f, c_i = 0.0f;
        Gate g{0.0f, 0.0f, 1.0f, 0.0f};
        if (in) {
          const float rv = Elem<T>::load(r + base + t);
          if constexpr ((RULE & kGateSoftplus) != 0) {
            softplus_pair(rv + rb, v, slope);
          } else {
            float comp;
            sigmoid_pair(rv, nrb, v, comp);
            slope = v * comp;
          }
          g = gate_of<RULE>(v, A2);
          if ((RULE & kGateSoftplus) != 0 && !(g.a > kMinNormal)) v = 0.0f;  // (as below)
          u = xv = Elem<T>::load(x + base + t);
          if constexpr (IG) {
            sigmoid_pair(Elem<T>::load(ig + base + t), nib, s_i, c_i);
            u *= s_i;
          }
        }
        const float q = g.w * u;
        if (!ahead && c < pieces - 1) from = enter[c][place];
        else enter[c][place] = from;
        auto step = [&](float h) { return apply_map<true>(cut ? 0.0f : g.a, q, h); };
        float hb = lanes_in_turn(lanes, from, step, [&](float h) {
          const float before = lane_before(h, from);
          return lane == 0 ? from : before;
        });
        const float h = step(hb);
        if (ahead) {
          from = __shfl(h, place | (lanes - 1));
          continue;
        }
        if (cut) hb = 0.0f;
        float dh = in ? Elem<T>::load(dy + base + t) : 0.0f;
        if constexpr (ZG) {
          if (in) {
            const float zv = Elem<T>::load(z + base + t);
            float s, c_z;
            sigmoid_pair(zv, 0.0f, s, c_z);
            const float ds = dh * s;
            Elem<T>::store(dz + base + t, ds * h * __builtin_fmaf(zv, c_z, 1.0f));
            dh = ds * zv;
          }
        }
        auto back = [&](float m) { return cut ? 0.0f : g.a * (dh + m); };
        const float m = lanes_in_turn(lanes, M, back, [&](float w) {
          const float after = lane_after(w, M);
          return at.last ? M : after;
        });
        M = __shfl(back(m), place & ~(lanes - 1));
        if (in) {  // the gradients of the step, as below
          const float lam = dh + m;
          float bend = g.a * u;
          if constexpr ((RULE & kGateUnit) != 0) bend = g.w > 0.0f ? bend * g.a * rcp_hw(g.w) : 0.0f;
          const float de = lam * __builtin_fmaf(g.a, hb, -bend);
          const float o = de * (slope * Ad);
          Elem<T>::store(dr + base + t, o);
          sA += (double)(de * v);
          srb += (double)o;
          float ox = lam * g.w;
          if constexpr (IG) {
            ox *= s_i;
            const float oi = ox * xv * c_i;
            Elem<T>::store(di + base + t, oi);
            sib += (double)oi;
          }
          Elem<T>::store(dx + base + t, ox);
        }
      }
    }
  };

  // whether the row cannot be composed
  auto must_turn = [&] {
    return grows_fast<RULE>(A2) && may_overflow<T, RULE, W>(r + base, A2, rb, at, p, s_most);
  };
  auto blocks = [&](int b0, int turn, auto whole, auto once) {
    constexpr bool WHOLE = decltype(whole)::value, ONCE = decltype(once)::value;
    const int blk = b0 + w0;  // past the last block: no steps, the identity
    const int64_t t0 = (int64_t)blk * kGatedBlock + lane * RN;
    const int64_t left = WHOLE ? kGatedBlock : at.live ? p.seqlen - t0 : 0;
    const RunWords<T> wr = ST::template load<ONCE>(r + base + t0, left), wx = ST::template load<ONCE>(x + base + t0, left);
    RunWords<T> wi, wz;
    if constexpr (IG) wi = ST::template load<ONCE>(ig + base + t0, left);
    if constexpr (ZG) wz = ST::template load<ONCE>(z + base + t0, left);
    const RunWords<T> wd = ST::template load<ONCE>(dy + base + t0, left);
    const bool packed = W == 0 || starts != nullptr;
    uint32_t cut = 0;
    if (starts != nullptr) cut = ST::starts(starts + (int64_t)b * p.seqlen + t0, left);
    const uint32_t in = WHOLE ? ~0u : ST::inside(left);
    const float H = WHOLE || blk < p.nblk ? ckpt[((int64_t)b * p.nblk + blk) * p.dim + d] : 0.0f;

    // g of each step, A dg/dr, the input gate and its complement
    float g[kRun], sA_[kRun], fx[kRun], gi[kRun], ci[kRun], a[kRun], w[kRun], q[kRun], dh[kRun];
    run_floats<T>(wr, g);
    run_floats<T>(wx, fx);
    run_floats<T>(wd, dh);
    if constexpr (IG) run_floats<T>(wi, gi);
    float S[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) S[h] = 0.0f;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      float v, slope;
      if constexpr ((RULE & kGateSoftplus) != 0) {
        softplus_pair(g[k] + rb, v, slope);
      } else {
        float c;
        sigmoid_pair(g[k], nrb, v, c);
        slope = v * c;
      }
      const Gate t = gate_of<RULE>(v, A2);
      // A softplus has no bound: where the decay is at its floor, g may be as far
      // above 1 as the floor is below it, and its product with the decay's gradient
      // (for dA) not the 0 that it is for a = 0.
      g[k] = (RULE & kGateSoftplus) == 0 || t.a > kMinNormal ? v : 0.0f;
      sA_[k] = slope * Ad;
      a[k] = t.a;
      w[k] = t.w;
      q[k] = t.w * fx[k];
      if constexpr (IG) {
        sigmoid_pair(gi[k], nib, gi[k], ci[k]);
        q[k] *= gi[k];
      }
      if (!WHOLE && !(in & (1u << k))) {
        a[k] = 1.0f;
        q[k] = 0.0f;
        g[k] = 0.0f;   // nothing is added to dA,
        sA_[k] = 0.0f;  // nor to dr_bias (x and so di are 0 already)
      } else {
        S[k / RN] += t.e2;
      }
    }
    float P[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h)
      P[h] = (cut >> (h * RN) & ((1u << RN) - 1u)) != 0 ? 0.0f : __builtin_fmaxf(exp2_hw(S[h]), kMinNormal);

    // the states: hb[k] before step k (0 at a start), q[k] after it
    float hb[kRun];
    auto rerun = [&](auto cuts) {
      constexpr bool CUT = decltype(cuts)::value;
      float from = H;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float Pf = P[h], Q = 0.0f;
#pragma unroll
        for (int k = h * RN; k < (h + 1) * RN; ++k)
          Q = apply_map<CUT>(CUT && (cut & (1u << k)) ? 0.0f : a[k], q[k], Q);
        if (W == 0 && lane == 0) {
          Q = apply_map<true>(Pf, Q, from);
          Pf = 0.0f;
        }
        wave_prefix<CUT>(Pf, Q);
        const float end = apply_map<CUT>(Pf, Q, from);
        float v = lane_before(end, from);
        if (W == 0 && lane == 0) v = from;
        if constexpr (NH > 1) from = lane_value(end, 63);
#pragma unroll
        for (int k = h * RN; k < (h + 1) * RN; ++k) {
          hb[k] = CUT && (cut & (1u << k)) ? 0.0f : v;
          q[k] = v = __builtin_fmaf(a[k], hb[k], q[k]);
        }
      }
    };
    if (packed) rerun(BoolC<true>{});
    else rerun(BoolC<false>{});

    // the output gate: dz, and dh = dy silu(z)
    if constexpr (ZG) {
      float fz[kRun], o[kRun];
      run_floats<T>(wz, fz);
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        float s, c;
        sigmoid_pair(fz[k], 0.0f, s, c);
        const float ds = dh[k] * s;
        o[k] = ds * q[k] * __builtin_fmaf(fz[k], c, 1.0f);
        dh[k] = ds * fz[k];
      }
      ST::store(dz + base + t0, left, o);
    }

    // the adjoint entering each run from the right: the runs of the last half
    // first, lanes mirrored
    float m_run[NH];
    auto back = [&](auto cuts) {
      constexpr bool CUT = decltype(cuts)::value;
      const int place = threadIdx.x & 63;
      float Pr[NH], Qr[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float Q = 0.0f;
#pragma unroll
        for (int k = (h + 1) * RN - 1; k >= h * RN; --k) Q = CUT && (cut & (1u << k)) ? 0.0f : a[k] * (dh[k] + Q);
        // in a shared wave the row's last lane applies its map to what enters
        if (W == 0 && at.last) Q = apply_map<true>(P[h], Q, M);
        Pr[h] = lane_mirror(W == 0 && at.last ? 0.0f : P[h], place);
        Qr[h] = lane_mirror(Q, place);
        wave_prefix<CUT>(Pr[h], Qr[h]);
      }
      float Pt = Pr[0], Qt = Qr[0];
      if constexpr (NH == 2) compose_map<CUT>(Pt, Qt, Pr[1], Qr[1]);
      float from = through_waves<CUT, W, true>(maps, turn, w0, Pt, Qt, M);
#pragma unroll
      for (int h = NH - 1; h >= 0; --h) {
        const float end = apply_map<CUT>(Pr[h], Qr[h], from);
        m_run[h] = lane_mirror(lane_before(end, from), place);
        if (W == 0 && at.last) m_run[h] = M;
        if constexpr (W == 0) M = lane_mirror(end, place);  // the first lane's goes to dh0
        else from = lane_value(end, 63);
      }
      if constexpr (W == 1) M = from;
    };
    if (packed) back(BoolC<true>{});
    else back(BoolC<false>{});

    // the gradients of each step, from the right; with u = x sigmoid(i)
    // de = lambda (a h_before - u (a or a^2/w)), the bracket's second term from
    // dw/de = -a, or -a^2/w (0 where w is 0)
    float odx[kRun], odr[kRun], odi[kRun];
    float pA = 0.0f, prb = 0.0f, pib = 0.0f;
#pragma unroll
    for (int k = kRun - 1; k >= 0; --k) {
      float& m = m_run[k / RN];
      const float lam = dh[k] + m;
      m = a[k] * lam;
      if (packed && (cut & (1u << k))) m = 0.0f;
      const float u = IG ? fx[k] * gi[k] : fx[k];
      float bend = a[k] * u;
      if constexpr ((RULE & kGateUnit) != 0) bend = w[k] > 0.0f ? bend * a[k] * rcp_hw(w[k]) : 0.0f;
      const float de = lam * __builtin_fmaf(a[k], hb[k], -bend);
      odr[k] = de * sA_[k];
      pA = __builtin_fmaf(de, g[k], pA);
      prb += odr[k];
      odx[k] = lam * w[k];
      if constexpr (IG) {
        odx[k] *= gi[k];
        odi[k] = odx[k] * fx[k] * ci[k];
        pib += odi[k];
      }
    }
    ST::store(dx + base + t0, left, odx);
    ST::store(dr + base + t0, left, odr);
    if constexpr (IG) ST::store(di + base + t0, left, odi);
    sA += (double)pA;
    srb += (double)prb;
    if constexpr (IG) sib += (double)pib;
  };
  if (must_turn()) {
    if (w0 == 0) in_turn();
  } else if constexpr (W == 0) {
    blocks(0, 0, BoolC<false>{}, BoolC<false>{});
  } else {
    int b0 = (p.nblk - 1) / W * W, turn = 0;
    if ((int64_t)(b0 + W) * kGatedBlock > p.seqlen) {
      blocks(b0, turn, BoolC<false>{}, BoolC<false>{});
      b0 -= W;
      turn ^= 1;
    }
    auto wholes = [&](auto once) {
      for (; b0 >= 0; b0 -= W, turn ^= 1) blocks(b0, turn, BoolC<true>{}, once);
    };
    if (p.once) wholes(BoolC<true>{});
    wholes(BoolC<false>{});
  }

  for (int off = 1; off < (W == 0 ? p.lanes : 64); off <<= 1) {
    sA += __shfl_xor(sA, off);
    srb += __shfl_xor(srb, off);
    if constexpr (IG) sib += __shfl_xor(sib, off);
  }
  if constexpr (W > 1) {
    __shared__ double s_sum[3][W];
    if (lane == 0) {
      s_sum[0][w0] = sA;
      s_sum[1][w0] = srb;
      s_sum[2][w0] = sib;
    }
    __syncthreads();
    sA = srb = sib = 0.0;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      sA += s_sum[0][j];
      srb += s_sum[1][j];
      sib += s_sum[2][j];
    }
  }
  if (lane == 0 && w0 == 0 && at.live) {
    row_dA[row] = (float)sA;
    if (row_drb != nullptr) row_drb[row] = (float)srb;
    if (IG && row_dib != nullptr) row_dib[row] = (float)sib;
    if (dh0 != nullptr) dh0[row] = M;
  }
}

// The rows' sums over the batch: out[k][d] = sum_b part[k][b][d], in float64 in
// the order of the batch.
__global__ __launch_bounds__(256) void gated_sum_kernel(const float* __restrict__ part, float* __restrict__ dA,
                                                        float* __restrict__ drb, float* __restrict__ dib,
                                                        int batch, int dim) {
  const int d = blockIdx.x * 256 + threadIdx.x;
  float* out = blockIdx.y == 0 ? dA : blockIdx.y == 1 ? drb : dib;
  if (d >= dim || out == nullptr) return;
  const float* p = part + (int64_t)blockIdx.y * batch * dim + d;
  double s = 0.0;
  for (int b = 0; b < batch; ++b) s += (double)p[(int64_t)b * dim];
  out[d] = (float)s;
}

// One token of every channel: a lane per channel.
template <typename T, int RULE, bool IG, bool ZG>
__global__ __launch_bounds__(256) void gated_step_kernel(
    const float* state, const T* __restrict__ x, const T* __restrict__ r, const float* __restrict__ A,
    const float* __restrict__ r_bias, const T* __restrict__ ig, const float* __restrict__ i_bias,
    const T* __restrict__ z, const uint8_t* __restrict__ starts, T* __restrict__ y, float* state_out, int b0,
    int dim) {
  const int d = blockIdx.x * 256 + threadIdx.x;
  if (d >= dim) return;
  const int b = b0 + (int)blockIdx.y;
  const int64_t at = (int64_t)b * dim + d;
  const float rb = r_bias != nullptr ? r_bias[d] : 0.0f;
  const Gate g = gate_of<RULE>(gate_value<RULE>(Elem<T>::load(r + at), rb, -rb * kLog2e), A[d] * kLog2e);
  float h = g.w * Elem<T>::load(x + at);
  if constexpr (IG) h *= sigmoid_f32(Elem<T>::load(ig + at), i_bias != nullptr ? -i_bias[d] * kLog2e : 0.0f);
  if (starts == nullptr || starts[b] == 0) h = __builtin_fmaf(g.a, state[at], h);
  state_out[at] = h;
  if constexpr (ZG) h *= silu_f32(Elem<T>::load(z + at));
  Elem<T>::store(y + at, h);
}

namespace {

// Calls f<RULE, IG, ZG> with the launch's rule and gates as constants.
template <typename F>
hipError_t by_rule(const GatedLaunch& a, F&& f) {
  auto gates = [&](auto rule) {
    constexpr int R = decltype(rule)::value;
    if (a.i != nullptr)
      return a.z != nullptr ? f.template operator()<R, true, true>() : f.template operator()<R, true, false>();
    return a.z != nullptr ? f.template operator()<R, false, true>() : f.template operator()<R, false, false>();
  };
  const int rule = (a.softplus ? kGateSoftplus : 0) | (a.unit ? kGateUnit : 0);
  switch (rule) {
    case 0: return gates(std::integral_constant<int, 0>{});
    case 1: return gates(std::integral_constant<int, 1>{});
    case 2: return gates(std::integral_constant<int, 2>{});
    default: return gates(std::integral_constant<int, 3>{});
  }
}

// Waves to a row: several rows to a wave up to half a wave's block (0); one where
// the rows alone make the 8192 waves that fill the chip (batch 8, dim 5120, L 2048,
// backward: 231 us, with four 257), more where they do not and the sequence has
// blocks for them (batch 3, dim 1000, L 1777 float32: one 23.4, four 22.6, sixteen 68;
// batch 1, dim 2048, L 65536 bf16: 266, 234, 238).  Sixteen for the fewest rows, by
// what it gives in long ones (batch 1, L 65536 bf16, both gates, forward and backward
// with sixteen, with four: dim 64 28 and 45 us, 41 and 65; dim 512 60 and 122, 61 and
// 121; dim 1500 179 and 345, 199 and 370); in short ones it costs (dim 1500, L 8192: 31
// and 52, 23 and 39; L 4096: 24 and 51, 13 and 23; dim 512 the same at both).
int waves_of(const GatedLaunch& a) {
  const int64_t rows = (int64_t)a.batch * a.dim, nblk = (a.seqlen + kGatedBlock - 1) / kGatedBlock;
  if (a.seqlen <= 256) return 0;
  if (rows >= 8192 || nblk == 1) return 1;
  return rows >= 2048 || nblk <= 4 ? 4 : 16;
}

// Whether inputs are read past the caches: rows of whole lines (others
// share lines between waves, which the caches then join) in a call whose tensors
// are twice the 256 MiB that the last cache may hold.  Batch 16, dim 5120, L 2048:
// 220 us so, 238 otherwise; batch 8, its backward: 201, 212; batch 4, dim 1000, L
// 8000, 320 MB of tensors again and again: 61, 52.
bool read_once(const GatedLaunch& a) {
  const int64_t streams = 3 + (a.i != nullptr) + (a.z != nullptr) + (a.dy != nullptr ? 2 + (a.i != nullptr) + (a.z != nullptr) : 0);
  const int64_t row = a.seqlen * (a.dtype == Dtype::BF16 ? 2 : 4), bytes = (int64_t)a.batch * a.dim * row;
  auto lines = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 128 == 0; };
  return row % 128 == 0 && streams * bytes > (int64_t)512 << 20 && lines(a.x) && lines(a.r) && lines(a.i) &&
         lines(a.z) && lines(a.dy);
}

GatedSizes sizes_of(const GatedLaunch& a) {
  int lanes = 64;
  if (waves_of(a) == 0) {
    lanes = 1;
    while (lanes * kRun < a.seqlen) lanes *= 2;
  }
  return GatedSizes{a.batch * a.dim, a.dim, (int)a.seqlen, (int)((a.seqlen + kGatedBlock - 1) / kGatedBlock), lanes,
                    read_once(a)};
}

// Workgroups: of rows that share waves, of a wave to a row, or a row each.
template <int W>
dim3 groups_of(const GatedSizes& s) {
  const int64_t rows = W == 0 ? (int64_t)group_waves(W) * 64 / s.lanes : W == 1 ? group_waves(W) : 1;
  return grid_of((s.rows + rows - 1) / rows, 64 * group_waves(W));
}

template <typename T>
struct FwdLaunch {
  const GatedLaunch& a;
  hipStream_t stream;
  template <int RULE, bool IG, bool ZG>
  hipError_t operator()() const {
    switch (waves_of(a)) {
      case 0: return launch<RULE, IG, ZG, 0>();
      case 1: return launch<RULE, IG, ZG, 1>();
      case 4: return launch<RULE, IG, ZG, 4>();
      default: return launch<RULE, IG, ZG, 16>();
    }
  }
  template <int RULE, bool IG, bool ZG, int W>
  hipError_t launch() const {
    const GatedSizes s = sizes_of(a);
    const dim3 grid = groups_of<W>(s);
    gated_fwd_kernel<T, RULE, IG, ZG, W><<<grid, 64 * group_waves(W), 0, stream>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.r), a.A, a.r_bias, static_cast<const T*>(a.i),
        a.i_bias, static_cast<const T*>(a.z), a.starts, a.h0, static_cast<T*>(a.y), a.last_state, a.ckpt, s);
    return hipGetLastError();
  }
};

template <typename T>
struct BwdLaunchOf {
  const GatedLaunch& a;
  hipStream_t stream;
  template <int RULE, bool IG, bool ZG>
  hipError_t operator()() const {
    switch (waves_of(a)) {
      case 0: return launch<RULE, IG, ZG, 0>();
      case 1: return launch<RULE, IG, ZG, 1>();
      case 4: return launch<RULE, IG, ZG, 4>();
      default: return launch<RULE, IG, ZG, 16>();
    }
  }
  template <int RULE, bool IG, bool ZG, int W>
  hipError_t launch() const {
    const GatedSizes s = sizes_of(a);
    const dim3 grid = groups_of<W>(s);
    // one row per channel: its sums are the results
    const bool direct = a.batch == 1;
    const int64_t plane = (int64_t)a.batch * a.dim;
    gated_bwd_kernel<T, RULE, IG, ZG, W><<<grid, 64 * group_waves(W), 0, stream>>>(
        static_cast<const T*>(a.x), static_cast<const T*>(a.r), a.A, a.r_bias, static_cast<const T*>(a.i),
        a.i_bias, static_cast<const T*>(a.z), a.starts, a.ckpt, static_cast<const T*>(a.dy), a.dlast,
        static_cast<T*>(a.dx), static_cast<T*>(a.dr), static_cast<T*>(a.di), static_cast<T*>(a.dz),
        direct ? a.dA : a.part, direct ? a.dr_bias : a.part + plane, direct ? a.di_bias : a.part + 2 * plane,
        a.dh0, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || direct) return e;
    gated_sum_kernel<<<dim3((unsigned)((a.dim + 255) / 256), IG ? 3 : 2), 256, 0, stream>>>(
        a.part, a.dA, a.dr_bias, a.di_bias, a.batch, a.dim);
    return hipGetLastError();
  }
};

template <typename T>
struct StepLaunch {
  const GatedLaunch& a;
  hipStream_t stream;
  template <int RULE, bool IG, bool ZG>
  hipError_t operator()() const {
    return by_row_slices(a.batch, hipSuccess, [&](int b0, int nb) {
      gated_step_kernel<T, RULE, IG, ZG><<<dim3((unsigned)((a.dim + 255) / 256), (unsigned)nb), 256, 0, stream>>>(
          a.h0, static_cast<const T*>(a.x), static_cast<const T*>(a.r), a.A, a.r_bias,
          static_cast<const T*>(a.i), a.i_bias, static_cast<const T*>(a.z), a.starts, static_cast<T*>(a.y),
          a.last_state, b0, a.dim);
      return hipGetLastError();
    });
  }
};

}  // namespace

hipError_t launch_gated_fwd(const GatedLaunch& a, hipStream_t stream) {
  return a.dtype == Dtype::BF16 ? by_rule(a, FwdLaunch<uint16_t>{a, stream}) : by_rule(a, FwdLaunch<float>{a, stream});
}

hipError_t launch_gated_bwd(const GatedLaunch& a, hipStream_t stream) {
  return a.dtype == Dtype::BF16 ? by_rule(a, BwdLaunchOf<uint16_t>{a, stream})
                                : by_rule(a, BwdLaunchOf<float>{a, stream});
}

hipError_t launch_gated_step(const GatedLaunch& a, hipStream_t stream) {
  return a.dtype == Dtype::BF16 ? by_rule(a, StepLaunch<uint16_t>{a, stream})
                                : by_rule(a, StepLaunch<float>{a, stream});
}

}  // namespace ssm
