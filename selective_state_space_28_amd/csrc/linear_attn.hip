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
// A workgroup of 4 waves owns a (batch row, head, segment) and 16 or 32 value columns for
// each of its waves.  S never leaves the matrix cores' accumulators.  16-bit operands use
// v_mfma_f32_16x16x32_bf16, float32 v_mfma_f32_16x16x4_f32.  HBM sees q, k, v and y once
// (and k and v once more where rows are split); batch 16, L 2048, 32 heads of 128, bf16:
// 290 to 335 us by the clock, 3.2 to 3.7 TB/s.  What bounds it there is the chain of a chunk, with two
// waves to a SIMD: VALUs busy 0.51 of the time (the parts of S and of the decayed v, the
// decay of S), matrix cores 0.34, LDS 0.33.  8 waves of 16 columns, four to a SIMD, spill or
// read LDS twice as often: 385 us for 327.
//
// Roundings with bf16 storage.  The decayed v, whose products with k make the float32
// state, goes in three parts, which is exact.  P as it meets V, and S as it meets q, go in
// two (2^-16): one part, rounded, would leave its 2^-9 in every output, for 295 us in place of 326
// (S) and 495 in place of 512 (P, batch 16, L 2048, 40 heads of 128).  The decay's
// gradient, a float32 output, has P, S and R in three parts each.
#include "linear_attn.hpp"
#include "runs.hpp"
#include "ssm_math.hpp"

namespace ssm {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) char lds_char;

// The compiler moves nothing over this: loads of later operands, moved up, would
// take registers that the state needs.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// A lane's number as a value of its own: LDS addresses formed from it, one
// instruction each, are neither formed before the loop nor shared with other code,
// and held in registers meanwhile.
__device__ __forceinline__ int own(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

constexpr int kWaves = 4;  // of a sweep's workgroup
constexpr int kThreads = 64 * kWaves;

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

// A tile in LDS, row-major, the 16-byte pieces of a row permuted by the row so that
// no access of the kernel meets a bank twice: 16 rows of one piece (operands
// contracted along the rows), 8 rows of two pieces (bf16, along the columns by
// transposing reads), 4 rows of four (float32, along the columns), whole rows
// (staging).
template <typename T, int W>
struct Tile {
  static constexpr int kPiece = 16 / (int)sizeof(T);  // elements
  static constexpr int kPieces = W / kPiece;
  __device__ __forceinline__ static int order(int row) {
    if constexpr (kPieces >= 16) {
      const int r = row & 15;
      return sizeof(T) == 2 ? ((r << 1) | (r >> 3)) & 15 : r;
    } else {
      const int r = (row >> 1) & 7;
      return sizeof(T) == 2 ? ((r << 1) | (r >> 2)) & 7 : r;
    }
  }
  __device__ __forceinline__ static int at(int row, int col) {
    return row * W + ((col / kPiece) ^ order(row)) * kPiece + col % kPiece;
  }
};

// The matrix cores' operands for storage type T.  A fragment is what a lane
// supplies of CK contracted elements: with q = lane / 16, m = lane % 16, of row (or
// column) m the elements 4 q + e and 16 + 4 q + e of 32 (bf16, e < 4) or 4 q + e of
// 16 (float32, four products): the order in which a product's result, D[4 q + r][m],
// r < 4, holds S.
template <typename T>
struct Mat;

template <>
struct Mat<uint16_t> {
  static constexpr int C = 64;    // steps of a chunk
  static constexpr int CK = 32;
  static constexpr int E = 8;     // elements of a fragment
  typedef bf16x8 Frag;
  __device__ __forceinline__ static f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // Contracted along the tile's rows: row r0 + m, columns from c0 on (r0 a multiple of 16,
  // c0 of CK).  A lane's place in a row of pieces is kept, and moved by c0's bits, which
  // its own do not touch.
  template <int W>
  __device__ __forceinline__ static int row_base(int lane) {
    return Tile<uint16_t, W>::at(lane & 15, 4 * (lane >> 4));
  }
  template <int W>
  __device__ __forceinline__ static Frag row(const uint16_t* tile, int base, int r0, int c0) {
    const uint2 a = *reinterpret_cast<const uint2*>(tile + (base ^ c0) + r0 * W);
    const uint2 b = *reinterpret_cast<const uint2*>(tile + (base ^ (c0 + 16)) + r0 * W);
    return __builtin_bit_cast(Frag, make_uint4(a.x, a.y, b.x, b.y));
  }
  // the same where both operands come from here: 8 q + e of 32, one access
  template <int W>
  __device__ __forceinline__ static int run_base(int lane) {
    return Tile<uint16_t, W>::at(lane & 15, 8 * (lane >> 4));
  }
  template <int W>
  __device__ __forceinline__ static Frag run(const uint16_t* tile, int base, int r0, int c0) {
    return *reinterpret_cast<const Frag*>(tile + (base ^ c0) + r0 * W);
  }
  // Contracted along its columns, from column c0 (a multiple of 16) on: the transposing read
  // gives 4 rows of a column to a lane.
  template <int W>
  __device__ __forceinline__ static int col_base(int lane) {
    return Tile<uint16_t, W>::at(4 * (lane >> 4) + ((lane & 15) >> 2), 4 * (lane & 3));
  }
  template <int W>
  __device__ __forceinline__ static Frag col(const uint16_t* tile, int base, int r0, int c0) {
    const uint16_t* p = tile + (base ^ c0) + r0 * W;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * W));
    const s16x4 ab[2] = {a, b};
    return __builtin_bit_cast(Frag, ab);
  }
  __device__ __forceinline__ static float at(const Frag& f, int e) { return (float)f[e]; }
  __device__ __forceinline__ static void zero(Frag& f, int e) { f[e] = (__bf16)0.0f; }
  __device__ __forceinline__ static void set(Frag& f, int e, float v) { f[e] = (__bf16)v; }
  // sum + 0 f: NaN if an element is not finite
  __device__ __forceinline__ static float times_zero(const Frag& f, float sum) {
    const bf16x2 nil = {(__bf16)0.0f, (__bf16)0.0f};
#pragma unroll
    for (int e = 0; e < E; e += 2) sum = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{f[e], f[e + 1]}, nil, sum, false);
    return sum;
  }
};

template <>
struct Mat<float> {
  static constexpr int C = 32;
  static constexpr int CK = 16;
  static constexpr int E = 4;
  typedef f32x4 Frag;
  __device__ __forceinline__ static f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
  }
  template <int W>
  __device__ __forceinline__ static int row_base(int lane) {
    return Tile<float, W>::at(lane & 15, 4 * (lane >> 4));
  }
  template <int W>
  __device__ __forceinline__ static Frag row(const float* tile, int base, int r0, int c0) {
    return *reinterpret_cast<const Frag*>(tile + (base ^ c0) + r0 * W);
  }
  template <int W>
  __device__ __forceinline__ static int run_base(int lane) {
    return row_base<W>(lane);
  }
  template <int W>
  __device__ __forceinline__ static Frag run(const float* tile, int base, int r0, int c0) {
    return row<W>(tile, base, r0, c0);
  }
  // (rows r0 + 4 q and the three after it: the order of their pieces differs in two bits)
  template <int W>
  __device__ __forceinline__ static int col_base(int lane) {
    return Tile<float, W>::at(4 * (lane >> 4), lane & 15);
  }
  template <int W>
  __device__ __forceinline__ static Frag col(const float* tile, int base, int r0, int c0) {
    const float* p = tile + r0 * W;
    Frag f;
#pragma unroll
    for (int r = 0; r < 4; ++r) f[r] = p[(base ^ c0 ^ (Tile<float, W>::order(r) * 4)) + r * W];
    return f;
  }
  __device__ __forceinline__ static float at(const Frag& f, int e) { return f[e]; }
  __device__ __forceinline__ static void zero(Frag& f, int e) { f[e] = 0.0f; }
  __device__ __forceinline__ static void set(Frag& f, int e, float v) { f[e] = v; }
  __device__ __forceinline__ static float times_zero(const Frag& f, float sum) {
#pragma unroll
    for (int e = 0; e < E; ++e) sum = __builtin_fmaf(f[e], 0.0f, sum);
    return sum;
  }
};

// The weight of what does not reach is +0, and of what does, however small, another: -0 where
// the product has underflowed.  (A NaN that such a decay meets stays one.)
__device__ __forceinline__ float reaching(float w) { return w == 0.0f ? -0.0f : w; }
__device__ __forceinline__ bool reaches(float w) { return __float_as_uint(w) != 0; }

// A fragment's elements that reach; the others are 0, NaN or not.
__device__ __forceinline__ uint4 weighed(const f32x4 (&w)[2]) {  // bf16: 8 halves
  const auto two = [](float a, float b) { return (reaches(a) ? 0xffffu : 0u) | (reaches(b) ? 0xffff0000u : 0u); };
  return make_uint4(two(w[0][0], w[0][1]), two(w[0][2], w[0][3]), two(w[1][0], w[1][1]), two(w[1][2], w[1][3]));
}
__device__ __forceinline__ uint4 weighed(const f32x4 (&w)[1]) {
  const auto one = [](float a) { return reaches(a) ? 0xffffffffu : 0u; };
  return make_uint4(one(w[0][0]), one(w[0][1]), one(w[0][2]), one(w[0][3]));
}
template <typename Frag>
__device__ __forceinline__ Frag only(uint4 mask, const Frag& f) {
  const uint4 v = __builtin_bit_cast(uint4, f);
  return __builtin_bit_cast(Frag, make_uint4(v.x & mask.x, v.y & mask.y, v.z & mask.z, v.w & mask.w));
}

// The step (of CK) that element e of a lane's fragment is, q4 = 4 (lane / 16).
__device__ __forceinline__ int step_of(int e, int q4) { return 16 * (e / 4) + q4 + e % 4; }

// A float32 as a sum of N bf16 fragments' elements: the leading bits cut off, what
// is left cut off again, the last rounded.  Three hold a float32 exactly, two to
// 2^-16.  (Of an infinite value the rest is NaN, and so is what it meets.)
__device__ __forceinline__ float cut16(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

// the upper halves of both, a's below: one instruction
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

template <typename T, int N>
struct Parts {
  typename Mat<T>::Frag f[N];
};

template <int N>
__device__ __forceinline__ Parts<uint16_t, N> parts_of(const float (&x)[8]) {
  Parts<uint16_t, N> p;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    float v0 = x[e], v1 = x[e + 1];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      bf16x2 hi = {(__bf16)v0, (__bf16)v1};
      if (k + 1 < N) {
        hi = __builtin_bit_cast(bf16x2, upper_halves(v0, v1));
        v0 -= cut16(v0);
        v1 -= cut16(v1);
      }
      p.f[k][e] = hi.x;
      p.f[k][e + 1] = hi.y;
    }
  }
  return p;
}

template <int N>
__device__ __forceinline__ Parts<float, 1> parts_of(const float (&x)[4]) {
  Parts<float, 1> p;
  p.f[0] = f32x4{x[0], x[1], x[2], x[3]};
  return p;
}

constexpr uint32_t kNowhere = 0x80000000u;  // an offset behind every extent

// ---- staging ----------------------------------------------------------------------
// Rows of a (batch, head) slice in the order of the sweep: step u at p + u * st bytes
// (st < 0 backward in time).
// (Odd widths: batch 3, 1777 steps, 10 heads of 50 and 100 in float32, packed: 132 us element
// by element, 92 by words.)
struct Slice {
  const char* p;
  int64_t st;
  int bytes;  // of a lane's copies: 16 or 4, as its alignment, strides and width are; 0: element by element
};

template <typename T>
__device__ __forceinline__ Slice slice_of(const AttnView& w, int64_t b, int h, int64_t first, int64_t dir, int width) {
  const uint64_t bits = reinterpret_cast<uintptr_t>(w.p) | (uint64_t)((w.sb | w.st | w.sh | (int64_t)width) * (int)sizeof(T));
  // (a chunk's offsets are 32 bits wide)
  const int bytes = w.st >= (int64_t)1 << 22 ? 0 : bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 0;
  return Slice{static_cast<const char*>(w.p) + (b * w.sb + (h / w.share) * w.sh + first * w.st) * (int64_t)sizeof(T),
               dir * w.st * (int64_t)sizeof(T), bytes};
}

// ROWS x W elements of a slice into LDS: zeros from column `width` and from row n on.
// The copies go past the registers, 1 KiB of LDS in one piece for a wave's access,
// whose lanes name what belongs there; an offset behind the extent gives zeros.
// They are under way until a wait for them.  Slices that cannot be read in vectors are
// copied element by element.
// (The wait stands for those that the compiler would set: 5 states between a vector
// instruction that writes a scalar register and the access that reads it, 1 after m0.)
__device__ __forceinline__ void copy_to_lds(uint32_t to, uint32_t at, u32x4_t buf, uint32_t base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(at), "s"(buf),
                 "s"(__builtin_amdgcn_readfirstlane(base))
               : "memory", "m0");
}

__device__ __forceinline__ void copy_word_to_lds(uint32_t to, uint32_t at, u32x4_t buf) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(at), "s"(buf)
               : "memory", "m0");
}

template <typename T, int ROWS, int W>
__device__ __forceinline__ void stage(T* lds, const Slice& s, int u, int width, int n, int wave) {
  using At = Tile<T, W>;
  constexpr int kAccesses = ROWS * W * (int)sizeof(T) / 1024 / kWaves;  // of a wave
  static_assert(kAccesses >= 1, "an access for every wave");
  const int lane = own(threadIdx.x & 63);
  if (s.bytes != 0) {
    // the lowest address first: row n - 1 backward in time
    const bool rev = s.st < 0;
    const uint32_t st = (uint32_t)(rev ? -s.st : s.st);
    const uint64_t low = reinterpret_cast<uint64_t>(s.p) + (uint64_t)((int64_t)(rev ? u + n - 1 : u) * s.st);
    u32x4_t buf;
    buf.x = __builtin_amdgcn_readfirstlane((uint32_t)low);
    buf.y = __builtin_amdgcn_readfirstlane((uint32_t)(low >> 32) & 0xffffu);
    buf.z = 0x7fffffffu;
    buf.w = 0x00020000u;
    const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char*)lds);
    // access k of a wave: rows kStep k and more, whose pieces are in one order for every k
    // (but with 32 and 64 pieces to a row)
    constexpr int kStep = ROWS / kAccesses;
    const int r0 = (wave * 64 + lane) / At::kPieces;
    if (s.bytes == 4) {  // 64 words of LDS for an access
      constexpr int kWord = 4 / (int)sizeof(T);  // elements
#pragma unroll 4
      for (int k = 0; k < 4 * kAccesses; ++k) {
        const int piece = ((k * kWaves + wave) * 64 + lane) >> 2;
        const int r = piece / At::kPieces, c = (piece % At::kPieces ^ At::order(r)) * At::kPiece + (lane & 3) * kWord;
        const uint32_t at = (uint32_t)(rev ? n - 1 - r : r) * st + (uint32_t)(c * (int)sizeof(T));
        copy_word_to_lds(to + (uint32_t)(k * kWaves + wave) * 256u, r < n && c < width ? at : kNowhere, buf);
      }
    } else if (n == ROWS) {
#pragma unroll
      for (int k = 0; k < kAccesses; ++k) {
        const int c = (lane % At::kPieces ^ At::order(r0 + k * kStep)) * At::kPiece;
        const uint32_t at = (uint32_t)(rev ? kStep - 1 - r0 : r0) * st + (uint32_t)(c * (int)sizeof(T));
        copy_to_lds(to + (uint32_t)(k * kWaves + wave) * 1024u, c < width ? at : kNowhere, buf,
                    (uint32_t)((rev ? kAccesses - 1 - k : k) * kStep) * st);
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < kAccesses; ++k) {
        const int r = r0 + k * kStep, c = (lane % At::kPieces ^ At::order(r)) * At::kPiece;
        const uint32_t at = (uint32_t)(rev ? n - 1 - r : r) * st + (uint32_t)(c * (int)sizeof(T));
        copy_to_lds(to + (uint32_t)(k * kWaves + wave) * 1024u, r < n && c < width ? at : kNowhere, buf, 0);
      }
    }
  } else {
#pragma unroll 1
    for (int i = own(threadIdx.x); i < ROWS * W; i += kThreads) {
      const int r = i / W, c = i % W;
      T e = (T)0;
      if (r < n && c < width) e = reinterpret_cast<const T*>(s.p + (int64_t)(u + r) * s.st)[c];
      lds[At::at(r, c)] = e;
    }
  }
}

// Where the elements of S lie in memory, (kd, vd) or turned: a lane's offset, and what
// is the same for every lane.  Rows and columns that pad S lie nowhere.
struct StateAt {
  int row0, col0, kd, vd, row_step, col_step;
  __device__ __forceinline__ StateAt(const AttnSweep& a, bool turned, int col, int row)
      : row0(row), col0(col), kd(a.kd), vd(a.vd), row_step(turned ? 1 : a.vd), col_step(turned ? a.kd : 1) {}
  __device__ __forceinline__ bool in(int row, int col) const { return row0 + row < kd && col0 + col < vd; }
  __device__ __forceinline__ uint32_t lane(int row, int col) const {
    return in(row, col) ? 4u * (uint32_t)(row0 * row_step + col0 * col_step) : kNowhere;
  }
  __device__ __forceinline__ uint32_t fixed(int row, int col) const {
    return 4u * (uint32_t)(row * row_step + col * col_step);
  }
};

}  // namespace

// Where the parts of P lie in LDS, each a tile of 64 columns: of bf16 the upper two of four
// blocks of 16 rows have 32 columns that are read, so two parts of them lie side by side, 32
// rows high, and the lower two blocks' parts below those.  (12 KiB for two parts: a CU keeps two
// workgroups at key and value heads of 128.)
template <typename T, int PARTS>
struct ScoreTiles {
  static constexpr int C = Mat<T>::C;
  static constexpr int kHalf = 32 * C, kUpper = (PARTS + 1) / 2;
  static constexpr int kSize = sizeof(T) == 2 ? (kUpper + PARTS) * kHalf : C * C;
  // the first row of a row block, and the first column
  __device__ __forceinline__ static int rows(int part, int it) {
    if (sizeof(T) == 4) return it * 16 * C;
    return it < 2 ? part / 2 * kHalf + it * 16 * C : (kUpper + part) * kHalf + (it - 2) * 16 * C;
  }
  __device__ __forceinline__ static int column(int part, int it) { return sizeof(T) == 2 && it < 2 ? 32 * (part & 1) : 0; }
};

// Tiles of P on and below the diagonal, row by row: 2 bits of each one's row and column.
__device__ __forceinline__ int tile_row(int tile) { return (0xffa94 >> (2 * tile)) & 3; }
__device__ __forceinline__ int tile_col(int tile) { return (0xe4910 >> (2 * tile)) & 3; }

// What a segment leaves of the state that enters it: e^{g steps}; -1 (nothing) where a
// sequence starts in it; and where a growing head's factor passes float32's range,
// minus its fourth root, more than 1: a state of 0 stays 0, and a small one need not overflow.
// (Four factors reach e^355: the smallest float passes the range before that.)
constexpr float kCut = -1.0f;
__device__ __forceinline__ float through_of(float g, int steps, bool cut) {
  const float t = decay_pow(g, (float)steps);
  return cut ? kCut : t == __builtin_inff() ? -decay_pow(g, 0.25f * (float)steps) : t;
}
__device__ __forceinline__ float carried(float t, float s, float added) {
  if (t == kCut) return added;
  if (t < kCut) return s == 0.0f ? added : __builtin_fmaf(s * t * t * t, t, added);
  return __builtin_fmaf(t, s, added);
}

enum AttnMode { kAttnOut = 0, kAttnSegments = 1, kAttnDecay = 2, kAttnDecaySegments = 3 };

// One workgroup: kWaves waves, CT tiles of 16 value columns each.  kAttnSegments: only
// the state that a segment adds, and what it leaves of the one before.  kAttnDecay:
// the forward sweep with R = dS/dg beside S, and dg = scale sum_t q_t R_t dy_t +
// <R_L, dlast>; R_u = e^g (R_{u-1} + S_{u-1}) gives, of a chunk,
//   diag(e^{g (i+1)}) Q (R + (i+1) S) + ((i-j) W o Q K^T) V
//   R <- e^{g C} (R + C S) + (diag((C-1-j) e^{g (C-1-j)}) K)^T V
// kAttnDecaySegments: what a segment adds to both.
//
// The next chunk's tiles are copied to LDS while this one is worked on: K, wanted to
// the end, into a second buffer, V and Q into their own once every wave has done with
// them.  (Through registers the state would not fit beside them.)
template <typename T, int KD, int CT, int MODE, bool PACKED>
__global__ __launch_bounds__(kThreads, KD <= 128 ? 2 : 1) void attn_sweep_kernel(const AttnSweeps all,
                                                                                const float* __restrict__ dlast,
                                                                                int64_t groups) {
  using M = Mat<T>;
  using Frag = typename M::Frag;
  constexpr int C = M::C, IT = C / 16, CK = M::CK, E = M::E;
  constexpr int NV = 16 * CT * kWaves;
  constexpr int KT = KD / 16;  // tiles of S above one another
  constexpr bool kSegments = MODE == kAttnSegments || MODE == kAttnDecaySegments;
  constexpr bool kDecay = MODE == kAttnDecay, kOut = !kSegments;
  constexpr bool kRate = kDecay || MODE == kAttnDecaySegments;  // R beside S
  constexpr int NU = sizeof(T) == 2 ? 3 : 1;  // parts of the decayed v, exact
  constexpr int NS = sizeof(T) == 2 ? kDecay ? 3 : 2 : 1;  // parts of S as an operand, exact or to 2^-16
  constexpr int kTiles = IT * (IT + 1) / 2;   // of P, on and below the diagonal
  constexpr int kMyTiles = (kTiles + kWaves - 1) / kWaves;
  constexpr int NP = NS;                      // parts of P, as S's
  using Scores = ScoreTiles<T, NP>;

  __shared__ __attribute__((aligned(16))) T s_q[kOut ? C * KD : 1];
  __shared__ __attribute__((aligned(16))) T s_keys[2][C * KD];
  __shared__ __attribute__((aligned(16))) T s_v[C * NV];
  __shared__ __attribute__((aligned(16))) T s_p[kOut ? Scores::kSize : 1];
  __shared__ __attribute__((aligned(16))) T s_dy[kDecay ? C * NV : 1];
  __shared__ float s_pw[C + 1];
  __shared__ __attribute__((aligned(16))) float s_enter[C], s_leave[C], s_left[kRate ? C : 1];
  __shared__ double s_sum[kWaves];

  int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int m = lane & 15, q4 = 4 * (lane >> 4);
  // consecutive workgroups go to the 8 dies in turn: a die takes consecutive numbers,
  // whose column blocks, and heads that share q, k or v, read the same lines
  int64_t id = group_index();
  const int64_t per = (groups + 7) / 8;
  id = (id & 7) * per + (id >> 3);
  if ((group_index() >> 3) >= per || id >= groups) return;
  const int64_t each = groups / all.n;
  const AttnSweep& a = all.s[id / each];
  id %= each;
  const int nvb = (a.vd + NV - 1) / NV;
  const int nsegs = kSegments ? a.nseg - 1 : a.nseg;
  const int vb = (int)(id % nvb);
  id /= nvb;
  const int h = (int)(id % a.heads);
  id /= a.heads;
  const int seg = (int)(id % nsegs), b = (int)(id / nsegs);

  const float g = a.g[h];
  const int L = (int)a.seqlen;
  const int len =
      a.lengths == nullptr ? L : __builtin_amdgcn_readfirstlane(min(max(a.lengths[b], 0), L));
  const int sh = a.rev ? 1 : 0;
  for (int i = threadIdx.x; i <= C; i += kThreads) s_pw[i] = decay_pow(g, (float)i);

  const int v0 = vb * NV;             // first value column of the workgroup
  const int vw = min(NV, a.vd - v0);  // its columns
  const int c0 = 16 * CT * wave;      // first of the wave, in the workgroup's
  const int64_t head = (int64_t)b * a.heads + h;
  const int64_t dir = a.rev ? -1 : 1, first = a.rev ? len - 1 : 0;
  const auto slice = [&](const AttnView& w, int width) { return slice_of<T>(w, b, h, first, dir, width); };
  const Slice sq = slice(a.q, a.kd), sk = slice(a.k, a.kd);
  Slice sv = slice(a.v, a.vd), sd{};
  sv.p += v0 * (int)sizeof(T);
  if constexpr (kDecay) {
    sd = slice(a.dy, a.vd);
    sd.p += v0 * (int)sizeof(T);
  }

  // S: rows 16 t + q4 + r, column v0 + c0 + 16 ct + m
  f32x4 S[CT][KT], R[kRate ? CT : 1][kRate ? KT : 1];
  const int64_t mat = (int64_t)a.kd * a.vd;
  const float* from = nullptr;
  if (kOut && seg > 0) from = a.seg_state + (head * a.nseg + seg) * mat;
  else if (kOut && a.state_in != nullptr) from = a.state_in + head * mat;
  const bool turned = kOut && a.transposed && seg == 0;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      S[ct][t] = f32x4{0, 0, 0, 0};
      if constexpr (kRate) R[ct][t] = f32x4{0, 0, 0, 0};
    }
  if (from != nullptr) {
    const Buf buf = make_buf(from, mat * 4);
    const StateAt at(a, turned, v0 + c0 + m, q4);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint32_t w[1];
          buf_load_words<1>(buf, at.lane(16 * t + r, 16 * ct), at.fixed(16 * t + r, 16 * ct), w);
          S[ct][t][r] = __uint_as_float(w[0]);
        }
  }
  if (kDecay && seg > 0) {
    const Buf buf = make_buf(a.seg_rate + (head * a.nseg + seg) * mat, mat * 4);
    const StateAt at(a, false, v0 + c0 + m, q4);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint32_t w[1];
          buf_load_words<1>(buf, at.lane(16 * t + r, 16 * ct), at.fixed(16 * t + r, 16 * ct), w);
          if constexpr (kRate) R[ct][t][r] = __uint_as_float(w[0]);
        }
  }
  if constexpr (kOut) {  // the masked halves of pairs of tiles stay zero
    for (int i = threadIdx.x; i < Scores::kSize; i += kThreads) s_p[i] = (T)0;
  }
  double dg = 0.0;
  bool cut = false;
  // whole chunks of whole columns are stored four columns at a time (offsets in 32 bits)
  const bool whole_out = vw == NV && a.vd % 4 == 0 && (sizeof(T) == 4 || !a.out_f32) &&
                         reinterpret_cast<uintptr_t>(a.out) % (4 * sizeof(T)) == 0 &&
                         (int64_t)a.heads * a.vd <= (int64_t)1 << 22;

  const int u_begin = (int)(seg * a.seglen);
  const int u_end = (int)min((int64_t)L, u_begin + a.seglen);
  T* out = static_cast<T*>(a.out);
  const auto valid = [&](int u) { return min(max(len - u, 0), C); };  // (u is at most seqlen + C, below 2^31)

  const auto there = [&](int u) { return u < u_end && u < len; };
  const auto stage_q = [&](int u) {
    if (kOut && there(u)) stage<T, C, KD>(s_q, sq, u, a.kd, valid(u), wave);
  };
  const auto stage_k = [&](int u, int into) {
    if (there(u)) stage<T, C, KD>(s_keys[into], sk, u, a.kd, valid(u), wave);
  };
  const auto stage_v = [&](int u) {
    if (there(u)) stage<T, C, NV>(s_v, sv, u, vw, valid(u), wave);
  };
  const auto stage_dy = [&](int u) {
    if constexpr (kDecay) {
      if (there(u)) stage<T, C, NV>(s_dy, sd, u, vw, valid(u), wave);
    }
  };
  stage_k(u_begin, 0);
  stage_q(u_begin);
  stage_v(u_begin);
  stage_dy(u_begin);
  int turn = 0;
  bool stored = false;

  // a lane's places in the tiles
  const int run_at = M::template run_base<KD>(lane), row_at = M::template row_base<KD>(lane),
            key_at = M::template col_base<KD>(lane), value_at = M::template col_base<NV>(lane) ^ c0,
            p_at = M::template row_base<C>(lane);
  // (where packed rows take registers too, what moves them is formed anew for every chunk)
  const auto place = [](int at) { return PACKED ? own(at) : at; };
  // this wave's tiles of P: e^{g (i-j)} of the lane's steps, 0 above the diagonal
  float wp[kOut ? kMyTiles : 1][4];
  if constexpr (kOut) {
#pragma unroll
    for (int k = 0; k < kMyTiles; ++k) {
      const int tile = min(wave + k * kWaves, kTiles - 1);
      const int apart = 16 * (tile_row(tile) - tile_col(tile)) + m - q4;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float n = (float)(apart - r);
        wp[k][r] = apart >= (kDecay ? r + 1 : r) ? reaching(decay_pow(g, n) * a.scale_p * (kDecay ? n : 1.0f)) : 0.0f;
      }
    }
  }

  // whether a sequence starts between this lane's step and the one before, a chunk ahead
  const auto starts_at = [&](int u0) {
    const int u = u0 + (threadIdx.x & 63);
    int f = 0;
    if (u < u_end && u < len && (int)(threadIdx.x & 63) < C && !(a.rev && u == 0))
      f = a.starts[(int64_t)b * L + (a.rev ? len - u : u)];
    return f;
  };
  int starts_here = 0;
  if constexpr (PACKED) starts_here = starts_at(u_begin);

  for (int u0 = u_begin; u0 < u_end; u0 += C) {
    const int n = valid(u0);
    if (n == 0 && MODE != kAttnOut) break;
    lane = own(lane);
    if (kOut && n == 0) {  // steps behind the row's length
      for (int64_t i = own(threadIdx.x); i < (int64_t)(u_end - u0) * vw; i += kThreads) {
        const int64_t at = (((int64_t)b * L + u0 + i / vw) * a.heads + h) * a.vd + v0 + i % vw;
        if (a.out_f32) static_cast<float*>(a.out)[at] = 0.0f;
        else out[at] = (T)0;
      }
      break;
    }
    // bit i: no state and no product crosses from step i-1 to step i
    const uint64_t B = PACKED ? __ballot(starts_here != 0) : 0;
    if constexpr (PACKED) starts_here = starts_at(u0 + C);
    const auto seen = [&](int i) { return __popcll(B & (~0ull >> (63 - i))); };  // starts up to and with step i
    const int total = seen(n - 1);

    // (the accesses of a wave end in the order in which they began: of those after its
    // copies, the stores of whole chunks, none is waited for)
    if (stored) asm volatile("s_waitcnt vmcnt(%0)" : : "n"(IT * CT) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    stored = false;
    __syncthreads();  // the tiles are there, and the chunk before is done with LDS
    const T* s_k = s_keys[turn];
    turn ^= 1;
    stage_k(u0 + C, turn);
    if (wave * 64 < C && own(threadIdx.x) < C) {  // the weights of the state that enters, and of each step in the one that leaves
      const int i = own(threadIdx.x), left = n - 1 - i;
      if constexpr (kOut) s_enter[i] = B == 0 || seen(i) == 0 ? reaching(s_pw[i + 1 - sh] * a.scale_in) : 0.0f;
      const float w = left >= 0 && (B == 0 || seen(i) == total) ? reaching(s_pw[left + sh] * a.scale_upd) : 0.0f;
      s_leave[i] = w;
      if constexpr (kRate) s_left[i] = w * (float)left;
    }

    // this wave's columns of V, contracted over the steps
    const int value_now = place(value_at), run_now = place(run_at);
    Frag vf[CT][C / CK];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int s = 0; s < C / CK; ++s) vf[ct][s] = M::template col<NV>(s_v, value_now, CK * s, 16 * ct);

    if constexpr (kOut) {
      // P = W o Q K^T, this wave's tiles, transposed so that a lane holds 4 steps j of a row i
      const int lane = own(threadIdx.x & 63), m = lane & 15, q4 = 4 * (lane >> 4);
      // (a wave without a last tile forms another's again, and keeps it to itself)
      int row0[kMyTiles], col0[kMyTiles];
      f32x4 tiles[kMyTiles];
      Frag fk[2][kMyTiles], fq[2][kMyTiles];
      int w0 = wave;
      asm volatile("" : "+s"(w0));  // (as `own`)
#pragma unroll
      for (int k = 0; k < kMyTiles; ++k) {
        const int tile = min(w0 + k * kWaves, kTiles - 1);
        row0[k] = 16 * tile_row(tile);
        col0[k] = 16 * tile_col(tile);
        tiles[k] = f32x4{0, 0, 0, 0};
        fk[0][k] = M::template run<KD>(s_k, run_now, col0[k], 0);
        fq[0][k] = M::template run<KD>(s_q, run_now, row0[k], 0);
      }
#pragma unroll
      for (int kk = 0; kk < KD / CK; ++kk) {
        in_order();
#pragma unroll
        for (int k = 0; k < kMyTiles; ++k) {
          if (kk + 1 < KD / CK) {
            fk[kk + 1 & 1][k] = M::template run<KD>(s_k, run_now, col0[k], (kk + 1) * CK);
            fq[kk + 1 & 1][k] = M::template run<KD>(s_q, run_now, row0[k], (kk + 1) * CK);
          }
          tiles[k] = M::mma(fk[kk & 1][k], fq[kk & 1][k], tiles[k]);
        }
      }
      in_order();
#pragma unroll
      for (int k = 0; k < kMyTiles; ++k) {
        if (w0 + k * kWaves >= kTiles) break;
        const f32x4 acc = tiles[k];
        const int it = row0[k] / 16, jt = col0[k] / 16;
        const int i = 16 * it + m;
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          bool kept = reaches(wp[k][r]);
          if (PACKED && B != 0) kept = kept && seen(i) == seen(16 * jt + q4 + r);
          p[r] = kept ? acc[r] * wp[k][r] : 0.0f;
        }
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int part = 0; part < NP; ++part) {
            T* to = s_p + Scores::rows(part, it) + Tile<T, C>::at(m, Scores::column(part, it) + 16 * jt + q4);
            uint2 w = make_uint2(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
            if (part + 1 < NP) {  // the upper halves, and what they leave
              w = make_uint2(upper_halves(p[0], p[1]), upper_halves(p[2], p[3]));
#pragma unroll
              for (int r = 0; r < 4; ++r) p[r] -= cut16(p[r]);
            }
            *reinterpret_cast<uint2*>(to) = w;
          }
        } else {
          *reinterpret_cast<f32x4*>(s_p + Tile<T, C>::at(i, 16 * jt + q4)) = f32x4{p[0], p[1], p[2], p[3]};
        }
      }
    }

    float odd = 0.0f;  // NaN if any of the values is not finite
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int s = 0; s < C / CK; ++s) odd = M::times_zero(vf[ct][s], odd);
    const bool careful = __any(!(odd == 0.0f));
    f32x4 acc[kOut ? CT : 1][kOut ? IT : 1], acc_r[kDecay ? CT : 1][kDecay ? IT : 1];
    if constexpr (kOut) {
      const int lane = own(threadIdx.x & 63);
      const f32x4 nil = {0, 0, 0, 0};
      const int row_now = place(row_at);
      // (Q S)^T: a lane holds 4 value columns of a step.  The next operands are on their way
      // while these are multiplied.
      constexpr int KK = KD / CK;
      Frag fq[2][IT];
      Parts<T, NS> ps[2][CT], pr[2][kDecay ? CT : 1];
      const auto operands = [&](int kk) {
#pragma unroll
        for (int it = 0; it < IT; ++it) fq[kk & 1][it] = M::template row<KD>(s_q, row_now, 16 * it, kk * CK);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          float sv[E], rv[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            sv[e] = S[ct][kk * (CK / 16) + e / 4][e % 4];
            if constexpr (kDecay) rv[e] = R[ct][kk * (CK / 16) + e / 4][e % 4];
          }
          ps[kk & 1][ct] = parts_of<NS>(sv);
          if constexpr (kDecay) pr[kk & 1][ct] = parts_of<NS>(rv);
        }
      };
      operands(0);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        in_order();
        if (kk + 1 < KK) operands(kk + 1);
#pragma unroll
        for (int k = 0; k < NS; ++k)
#pragma unroll
          for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
              acc[ct][it] = M::mma(ps[kk & 1][ct].f[k], fq[kk & 1][it], kk == 0 && k == 0 ? nil : acc[ct][it]);
              if constexpr (kDecay)
                acc_r[ct][it] = M::mma(pr[kk & 1][ct].f[k], fq[kk & 1][it], kk == 0 && k == 0 ? nil : acc_r[ct][it]);
            }
      }
    }
    __syncthreads();  // P and the weights are there, Q has been read, V is in registers
    stage_q(u0 + C);
    stage_v(u0 + C);
    {
      if constexpr (kOut) {
        const int lane = own(threadIdx.x & 63), m = lane & 15, q4 = 4 * (lane >> 4);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const int i = 16 * it + m;
          const float w = s_enter[i];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float o = acc[ct][it][r];
              if constexpr (kDecay) o = __builtin_fmaf(o, (float)(i + 1), acc_r[ct][it][r]);
              acc[ct][it][r] = PACKED && !reaches(w) ? 0.0f : o * w;
            }
        }
        in_order();
        const int p_now = place(p_at);
        // P V, of the values `of` gives
        const auto product = [&](auto of) {
#pragma unroll
          for (int s = 0; s < C / CK; ++s)
#pragma unroll
            for (int it = 0; it < IT; ++it) {
              if (CK * s >= 16 * (it + 1)) continue;
#pragma unroll
              for (int part = 0; part < NP; ++part) {
                const Frag fp =
                    M::template row<C>(s_p + Scores::rows(part, it), p_now, 0, Scores::column(part, it) + CK * s);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) acc[ct][it] = M::mma(of(vf[ct][s]), fp, acc[ct][it]);
              }
            }
        };
        if (!careful) {
          product([](const Frag& f) { return f; });
        } else {
          // Values that are not finite are left out: the zeros of P above its diagonal would
          // spread them.  Products of ones in their places with ones where P has its steps
          // count what each output takes of them: those are NaN.
          product([](Frag f) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (!finite_f32(M::at(f, e))) M::zero(f, e);
            return f;
          });
#pragma unroll
          for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int s = 0; s < C / CK; ++s) {
              if (CK * s >= 16 * (it + 1)) continue;
              in_order();
              const int i = 16 * it + m;
              Frag taken, one;
#pragma unroll
              for (int e = 0; e < E; ++e) {
                const int j = CK * s + step_of(e, q4);
                M::set(taken, e, j <= i && (!PACKED || seen(i) == seen(j)) ? 1.0f : 0.0f);
              }
#pragma unroll
              for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
                for (int e = 0; e < E; ++e) M::set(one, e, finite_f32(M::at(vf[ct][s], e)) ? 0.0f : 1.0f);
                const f32x4 bad = M::mma(one, taken, f32x4{0, 0, 0, 0});
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[ct][it][r] = bad[r] != 0.0f ? __builtin_nanf("") : acc[ct][it][r];
              }
            }
        }
        if constexpr (kDecay) {
          float sum = 0.0f;
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int i = 16 * it + m, c = c0 + 16 * ct + q4 + r;
                if (i < n && c < vw)
                  sum = __builtin_fmaf(acc[ct][it][r], Elem<T>::load(s_dy + Tile<T, NV>::at(i, c)), sum);
              }
          dg += (double)sum;
        } else if (whole_out && n == C) {
          stored = true;
          // the chunk's lowest row first
          const int64_t t0 = a.rev ? len - C - u0 : u0;
          const Buf buf = make_buf(out + (((int64_t)b * L + t0) * a.heads + h) * a.vd + v0, 0x7fffffff);
          const uint32_t step = (uint32_t)(a.heads * a.vd) * (uint32_t)sizeof(T);
#pragma unroll
          for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
              const uint32_t at =
                  (uint32_t)(a.rev ? C - 1 - 16 * it - m : 16 * it + m) * step + (uint32_t)(c0 + 16 * ct + q4) * (uint32_t)sizeof(T);
              const f32x4 o = acc[ct][it];
              if constexpr (sizeof(T) == 2) {
                const uint32_t words[2] = {pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
                buf_store_words<2>(buf, at, 0, words);
              } else {
                const uint32_t words[4] = {__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]),
                                           __float_as_uint(o[3])};
                buf_store_words<4>(buf, at, 0, words);
              }
            }
        } else {
#pragma unroll
          for (int it = 0; it < IT; ++it) {
            const int i = 16 * it + m, u = u0 + i;
            if (u >= u_end) continue;
            const int t = u < len && a.rev ? len - 1 - u : u;
            const int64_t at = (((int64_t)b * L + t) * a.heads + h) * a.vd + v0;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int c = c0 + 16 * ct + q4 + r;
                const float o = i < n ? acc[ct][it][r] : 0.0f;
                if (c < vw) {
                  if (a.out_f32) static_cast<float*>(a.out)[at + c] = o;
                  else Elem<T>::store(out + at + c, o);
                }
              }
          }
        }
      }

      in_order();
      if constexpr (kDecay) {
        __syncthreads();  // dy has been read
        stage_dy(u0 + C);
      }
      const int lane = own(threadIdx.x & 63), q4 = 4 * (lane >> 4);
      // the state behind the chunk
      const float pass = s_pw[n];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if constexpr (kRate) {
              R[ct][t][r] = __builtin_fmaf(S[ct][t][r], (float)n, R[ct][t][r]) * pass;
              if (PACKED && total != 0) R[ct][t][r] = 0.0f;
            }
            S[ct][t][r] *= pass;
            if (PACKED && total != 0) S[ct][t][r] = 0.0f;
          }
      const int key_now = place(key_at);
      constexpr int TT = 4;  // tiles at a time: products that do not wait for one another
      constexpr int kGroups = KT / TT;
      Parts<T, NU> px[CT], px2[kRate ? CT : 1];
      Frag kf[2][TT];
      const auto keys = [&](int i) {  // group i: steps CK (i / kGroups), tiles TT (i % kGroups)
        const int s = i / kGroups, t = i % kGroups * TT;
#pragma unroll
        for (int j = 0; j < TT; ++j) kf[i & 1][j] = M::template col<KD>(s_k, key_now, CK * s, 16 * (t + j));
      };
      uint4 taken = make_uint4(0, 0, 0, 0);  // packed rows: the steps that reach the state, not even a NaN of the others
      const auto values = [&](int s) {
        f32x4 w[E / 4], w2[E / 4];
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          w[e / 4] = *reinterpret_cast<const f32x4*>(s_leave + CK * s + step_of(e, q4));
          if constexpr (kRate) w2[e / 4] = *reinterpret_cast<const f32x4*>(s_left + CK * s + step_of(e, q4));
        }
        if constexpr (PACKED) taken = weighed(w);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          float x[E], x2[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float v = M::at(PACKED ? only(taken, vf[ct][s]) : vf[ct][s], e);
            x[e] = v * w[e / 4][e % 4];
            if constexpr (kRate) x2[e] = v * w2[e / 4][e % 4];
          }
          px[ct] = parts_of<NU>(x);
          if constexpr (kRate) px2[ct] = parts_of<NU>(x2);
        }
      };
      keys(0);
#pragma unroll
      for (int i = 0; i < kGroups * (C / CK); ++i) {
        const int t = i % kGroups * TT;
        if (t == 0) values(i / kGroups);
        in_order();
        if (i + 1 < kGroups * (C / CK)) keys(i + 1);
        if constexpr (PACKED) {
#pragma unroll
          for (int j = 0; j < TT; ++j) kf[i & 1][j] = only(taken, kf[i & 1][j]);
        }
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
          for (int j = 0; j < TT; ++j)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
              S[ct][t + j] = M::mma(kf[i & 1][j], px[ct].f[k], S[ct][t + j]);
              if constexpr (kRate) R[ct][t + j] = M::mma(kf[i & 1][j], px2[ct].f[k], R[ct][t + j]);
            }
      }
    }
    if (kSegments) cut |= B != 0;
  }

  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // no copy to LDS outlives the workgroup
  lane = own(lane);
  m = lane & 15;
  q4 = 4 * (lane >> 4);
  if constexpr (kSegments) {
    const int steps = min(max(len - u_begin, 0), u_end - u_begin);
    if (vb == 0 && threadIdx.x == 0) {
      a.seg_through[head * a.nseg + seg] = through_of(g, steps, cut);
      if constexpr (kRate) a.seg_steps[head * a.nseg + seg] = (float)steps;
    }
  } else if constexpr (MODE == kAttnDecay) {
    float sum = 0.0f;
    if (dlast != nullptr && seg == a.nseg - 1) {
      const Buf buf = make_buf(dlast + head * mat, mat * 4);
      const StateAt at(a, false, v0 + c0 + m, q4);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            uint32_t w[1];
            buf_load_words<1>(buf, at.lane(16 * t + r, 16 * ct), at.fixed(16 * t + r, 16 * ct), w);
            if (at.in(16 * t + r, 16 * ct)) sum = __builtin_fmaf(R[ct][t][r], __uint_as_float(w[0]), sum);
          }
    }
    dg = wave_sum(dg + (double)sum);
    if (lane == 0) s_sum[wave] = dg;
    __syncthreads();
    if (threadIdx.x == 0)
      a.part[(((int64_t)h * a.batch + b) * nvb + vb) * a.nseg + seg] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
    return;
  }
  float* to = nullptr;
  if (kSegments) to = a.seg_state + (head * a.nseg + seg + 1) * mat;
  else if (a.state_out != nullptr && seg == a.nseg - 1) to = a.state_out + head * mat;
  if (to == nullptr) return;
  // backward in time nothing passes a first step that starts a sequence
  const bool gone = MODE == kAttnOut && a.rev && a.starts != nullptr && len > 0 && a.starts[(int64_t)b * L] != 0;
  const Buf buf = make_buf(to, mat * 4);
  const StateAt at(a, MODE == kAttnOut && a.transposed, v0 + c0 + m, q4);
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t w[1] = {gone ? 0u : __float_as_uint(S[ct][t][r])};
        buf_store_words<1>(buf, at.lane(16 * t + r, 16 * ct), at.fixed(16 * t + r, 16 * ct), w);
      }
  if constexpr (MODE == kAttnDecaySegments) {
    const Buf rate = make_buf(a.seg_rate + (head * a.nseg + seg + 1) * mat, mat * 4);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t w[1] = {__float_as_uint(R[ct][t][r])};
          buf_store_words<1>(rate, at.lane(16 * t + r, 16 * ct), at.fixed(16 * t + r, 16 * ct), w);
        }
  }
}

// The states entering the segments from what each adds: S <- through S + added, and with
// `rate`, R <- through (R + steps S) + added; a thread an element.
__global__ __launch_bounds__(256) void attn_carry_kernel(const AttnSweeps all, bool rates, int64_t n) {
  int64_t i = group_index() * 256 + threadIdx.x;
  if (i >= n * all.n) return;
  const AttnSweep& a = all.s[i / n];
  i %= n;
  const int mat = a.kd * a.vd, nseg = a.nseg;
  float *state = a.seg_state, *rate = rates ? a.seg_rate : nullptr;
  const float *state_in = a.state_in, *steps = a.seg_steps;
  const int64_t head = i / mat;
  const int e = (int)(i - head * mat), row = e / a.vd, col = e - row * a.vd;
  float s = 0.0f, r = 0.0f;
  if (state_in != nullptr) s = state_in[head * mat + (a.transposed ? col * a.kd + row : e)];
  const int64_t first = head * nseg * mat + e;
  const float* th = a.seg_through + head * nseg;
  constexpr int U = 8;  // segments on their way at once
  for (int k0 = 0; k0 + 1 < nseg; k0 += U) {
    float added[U], more[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = k0 + u + 1 < nseg;
      added[u] = in ? state[first + (int64_t)(k0 + u + 1) * mat] : 0.0f;
      more[u] = in && rate != nullptr ? rate[first + (int64_t)(k0 + u + 1) * mat] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u;
      if (k + 1 >= nseg) break;
      const float t = th[k];
      if (rate != nullptr) {
        r = carried(t, __builtin_fmaf(steps[head * nseg + k], s, r), more[u]);
        rate[first + (int64_t)(k + 1) * mat] = r;
      }
      s = carried(t, s, added[u]);
      state[first + (int64_t)(k + 1) * mat] = s;
    }
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
                                                            int64_t per, int heads) {
  const int64_t h = group_index();
  if (h >= heads) return;
  const double* p = part + h * per;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < per; i += 64) s += p[i];
  s = wave_sum(s);
  if (threadIdx.x == 0) out[h] = (float)s;
}

// One token: S <- e^g S + k v^T, y = scale q S, bound by the state, read and written
// once (256 rows of 40 heads of 128 x 128: 235 us, 5.7 TB/s; a column a lane and a row at a
// time took 520).  A workgroup takes a (batch row, head) and kStepColumns value columns; V columns
// lie side by side in a lane (4, where rows of S are aligned so, or 1), so a row takes
// kStepColumns / V lanes, and a lane has kStepRows of its rows on their way at once.
constexpr int kStepColumns = 64, kStepRows = 8;

template <typename T, int V>
__global__ __launch_bounds__(256) void attn_step_kernel(const AttnStep a) {
  typedef float vecf __attribute__((ext_vector_type(V)));
  constexpr int kLanes = kStepColumns / V, kRows = 256 / kLanes;  // rows of S side by side
  __shared__ float s_k[kAttnMaxWidth], s_q[kAttnMaxWidth];
  __shared__ float s_y[kRows][kStepColumns + 4];
  const int lane = threadIdx.x % kLanes, row0 = threadIdx.x / kLanes;
  const int nvb = (a.vd + kStepColumns - 1) / kStepColumns;
  int64_t id = group_index();
  if (id >= (int64_t)a.batch * a.heads * nvb) return;
  const int vb = (int)(id % nvb);
  id /= nvb;
  const int h = (int)(id % a.heads), b = (int)(id / a.heads);
  const int col = vb * kStepColumns + lane * V;
  const auto base = [&](const AttnView& w) { return static_cast<const T*>(w.p) + b * w.sb + (h / w.share) * w.sh; };
  const T *pq = base(a.q), *pk = base(a.k), *pv = base(a.v);
  const bool first = a.starts != nullptr && a.starts[b] != 0;
  const int64_t at = ((int64_t)b * a.heads + h) * a.kd * a.vd + col;
  const bool in = col < a.vd;
  vecf s[kStepRows];
  const auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kStepRows; ++u) {
      const int row = r0 + u * kRows;
      if (in && !first && row < a.kd) s[u] = *reinterpret_cast<const vecf*>(a.state + at + (int64_t)row * a.vd);
      else s[u] = 0.0f;
    }
  };
  load(row0);
  if (threadIdx.x < a.kd) {
    s_k[threadIdx.x] = Elem<T>::load(pk + threadIdx.x);
    s_q[threadIdx.x] = Elem<T>::load(pq + threadIdx.x);
  }
  vecf v, y = 0.0f;
#pragma unroll
  for (int c = 0; c < V; ++c) v[c] = in ? Elem<T>::load(pv + col + c) : 0.0f;
  const float decay = decay_pow(a.g[h], 1.0f);
  __syncthreads();
  for (int r0 = row0; r0 < a.kd; r0 += kRows * kStepRows) {
    if (r0 != row0) load(r0);
#pragma unroll
    for (int u = 0; u < kStepRows; ++u) {
      const int row = r0 + u * kRows;
      if (!in || row >= a.kd) continue;
      const float k = s_k[row], q = s_q[row];
      vecf n;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float kv = k * v[c];
        n[c] = first ? kv : __builtin_fmaf(decay, s[u][c], kv);
        y[c] = __builtin_fmaf(q, n[c], y[c]);
      }
      *reinterpret_cast<vecf*>(a.state_out + at + (int64_t)row * a.vd) = n;
    }
  }
#pragma unroll
  for (int c = 0; c < V; ++c) s_y[row0][lane * V + c] = y[c];
  __syncthreads();
  const int c = vb * kStepColumns + (int)threadIdx.x;
  if (threadIdx.x < kStepColumns && c < a.vd) {
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) sum += s_y[r][threadIdx.x];
    Elem<T>::store(static_cast<T*>(a.y) + ((int64_t)b * a.heads + h) * a.vd + c, sum * a.scale);
  }
}

namespace {

// Tiles of value columns of a wave: 128 columns to a workgroup, or 64 (heads of up to 64
// values would leave half of them idle; of wider ones two tiles share what a wave reads
// of Q, K and P: batch 16, L 2048, 32 heads of 128 bf16 take 330 us with two, as much work in
// 64 heads of 64 values takes 410).
int column_tiles(int vd) { return vd <= 64 ? 1 : 2; }

template <typename T, int KD, int CT, int MODE>
hipError_t sweep(const AttnSweeps& all, const float* dlast, hipStream_t stream) {
  const AttnSweep& a = all.s[0];  // the others have its numbers of groups
  const int nvb = (a.vd + 64 * CT - 1) / (64 * CT);
  const int nsegs = MODE == kAttnSegments || MODE == kAttnDecaySegments ? a.nseg - 1 : a.nseg;
  const int64_t groups = (int64_t)all.n * a.batch * a.heads * nvb * nsegs;
  const dim3 grid = grid_of((groups + 7) / 8 * 8, kThreads);
  if (a.starts != nullptr) attn_sweep_kernel<T, KD, CT, MODE, true><<<grid, kThreads, 0, stream>>>(all, dlast, groups);
  else attn_sweep_kernel<T, KD, CT, MODE, false><<<grid, kThreads, 0, stream>>>(all, dlast, groups);
  return hipGetLastError();
}

template <typename T, int CT, int MODE>
hipError_t sweep_of(const AttnSweeps& all, const float* dlast, hipStream_t stream) {
  if (all.s[0].kd <= 64) return sweep<T, 64, CT, MODE>(all, dlast, stream);
  if (all.s[0].kd <= 128) return sweep<T, 128, CT, MODE>(all, dlast, stream);
  return sweep<T, 256, CT, MODE>(all, dlast, stream);
}

template <typename T, int MODE>
hipError_t sweep_of(const AttnSweeps& all, hipStream_t stream) {
  return column_tiles(all.s[0].vd) == 1 ? sweep_of<T, 1, MODE>(all, nullptr, stream)
                                        : sweep_of<T, 2, MODE>(all, nullptr, stream);
}

hipError_t carry(const AttnSweeps& all, bool rates, hipStream_t stream) {
  const AttnSweep& a = all.s[0];
  const int64_t n = (int64_t)a.batch * a.heads * a.kd * a.vd;
  attn_carry_kernel<<<grid_of((n * all.n + 255) / 256, 256), 256, 0, stream>>>(all, rates, n);
  return hipGetLastError();
}

template <typename T>
hipError_t run_sweeps(const AttnSweeps& all, hipStream_t stream) {
  if (all.s[0].nseg > 1) {
    hipError_t e = sweep_of<T, kAttnSegments>(all, stream);
    if (e == hipSuccess) e = carry(all, false, stream);
    if (e != hipSuccess) return e;
  }
  return sweep_of<T, kAttnOut>(all, stream);
}

template <typename T>
hipError_t run_decay(const AttnSweeps& all, const float* dlast, hipStream_t stream) {
  if (all.s[0].nseg > 1) {
    hipError_t e = sweep_of<T, 1, kAttnDecaySegments>(all, dlast, stream);
    if (e == hipSuccess) e = carry(all, true, stream);
    if (e != hipSuccess) return e;
  }
  return sweep_of<T, 1, kAttnDecay>(all, dlast, stream);
}

}  // namespace

int attn_column_blocks(int vd) { return (vd + 64 * column_tiles(vd) - 1) / (64 * column_tiles(vd)); }

int attn_decay_blocks(int vd) { return (vd + 63) / 64; }

// Workgroups and segments.  A sweep of one chunk after another takes a time that a CU's
// two workgroups share only in part (bf16, heads of 128, microseconds for 64 steps): 5.4 where
// half the CUs have one, 6.3 with one on each, 8.9 with two; float32, on its own matrix
// cores, 2.4 times as much.  Segments fill the CUs, and cost the pass that finds their states
// (0.58 of the main one's time) with two more launches and the states' traffic, some 20 us and
// more.  The least of these sums is taken, of up to 64 segments (batch 8, L 2048 bf16: 16 heads
// 182 us in one piece, 137 in segments; 32 heads 203 and 244; one row of 512 steps, 12 heads,
// float32: 112 and 45).  The same times are taken for the kernels that have one workgroup to a CU
// (key heads above 128; the decay's gradient of bf16 key heads above 64), whose 257 to 512
// workgroups are two rounds and are counted as one.
AttnSplit attn_split(int64_t groups, int64_t seqlen, int64_t state_elements, Dtype dtype) {
  const int64_t chunks = (seqlen + kAttnChunk - 1) / kAttnChunk;
  const double slower = dtype == Dtype::F32 ? 2.4 : 1.0;
  const auto rounds = [&](int64_t g) {
    const int64_t left = g % 512;
    return slower * (8.9 * (double)(g / 512) + (left == 0 ? 0.0 : left <= 128 ? 5.4 : left <= 256 ? 6.3 : 8.9));
  };
  AttnSplit best{1, (chunks > 0 ? chunks : 1) * kAttnChunk};
  if (groups <= 0) return best;
  double least = (double)chunks * rounds(groups);
  for (int64_t n = 2; n <= 64 && n <= chunks; ++n) {
    const int64_t per = (chunks + n - 1) / n, nseg = (chunks + per - 1) / per;
    const double states = 16e-6 / 4.0 * (double)state_elements * (double)nseg;  // four passes of float32 at 4 TB/s
    const double t = (double)per * (rounds(groups * nseg) + 0.58 * rounds(groups * (nseg - 1))) + 20.0 + states;
    if (t < least) {
      least = t;
      best = AttnSplit{(int)nseg, per * kAttnChunk};
    }
  }
  return best;
}

bool attn_alike(int a, int b) {
  const auto kind = [](int width) { return width <= 64 ? 0 : width <= 128 ? 1 : 2; };
  return kind(a) == kind(b);
}

hipError_t launch_attn_sweeps(const AttnSweeps& all, hipStream_t stream) {
  return all.s[0].dtype == Dtype::BF16 ? run_sweeps<uint16_t>(all, stream) : run_sweeps<float>(all, stream);
}

hipError_t launch_attn_decay_grad(const AttnSweep& a, const float* dlast, float* dlog_decay, hipStream_t stream) {
  AttnSweeps all{};
  all.s[0] = a;
  all.n = 1;
  const hipError_t e = a.dtype == Dtype::BF16 ? run_decay<uint16_t>(all, dlast, stream) : run_decay<float>(all, dlast, stream);
  if (e != hipSuccess) return e;
  attn_decay_sum_kernel<<<grid_of(a.heads, 64), 64, 0, stream>>>(
      a.part, dlog_decay, (int64_t)a.batch * attn_decay_blocks(a.vd) * a.nseg, a.heads);
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

namespace {

template <typename T>
hipError_t step(const AttnStep& a, hipStream_t stream) {
  const int64_t groups = (int64_t)a.batch * a.heads * ((a.vd + kStepColumns - 1) / kStepColumns);
  const dim3 grid = grid_of(groups, 256);
  const bool vec = a.vd % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) | reinterpret_cast<uintptr_t>(a.state_out)) % 16 == 0;
  if (vec) attn_step_kernel<T, 4><<<grid, 256, 0, stream>>>(a);
  else attn_step_kernel<T, 1><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_step(const AttnStep& a, hipStream_t stream) {
  return a.dtype == Dtype::BF16 ? step<uint16_t>(a, stream) : step<float>(a, stream);
}

}  // namespace ssm
