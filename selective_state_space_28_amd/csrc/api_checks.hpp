// api_checks.hpp -- argument checks that every entry point of the C ABI makes
// before its first HIP call: alignment, byte ranges and sizes.
#pragma once

#include <climits>
#include <cstddef>
#include <cstdint>

#include "ssm.h"

namespace ssm {

inline int elem_bytes(int dtype) { return dtype == SSM_BF16 ? 2 : 4; }

inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }

inline bool aligned(const void* p, size_t a) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The byte range [lo, hi) a buffer occupies; a null pointer or zero bytes
// occupies none.  Aliasing is judged on these ranges, not on pointer
// equality, so an output that starts inside an input (or ends inside one) is
// rejected too.
struct Span {
  uintptr_t lo, hi;
};

inline Span span(const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (p == nullptr || bytes == 0) return Span{0, 0};
  return Span{lo, lo + bytes};
}

inline bool overlap(const Span& a, const Span& b) {
  return a.hi > a.lo && b.hi > b.lo && a.lo < b.hi && b.lo < a.hi;
}

// Whether a buffer the call writes overlaps another buffer the call writes,
// or one it reads.  Inputs may overlap each other (they are only read).
template <size_t NO, size_t NI>
bool writes_overlap(const Span (&outs)[NO], const Span (&ins)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (size_t j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return true;
  }
  return false;
}

// The scan kernels keep step positions in 32 bits.
constexpr int64_t kMaxSeqlen = INT32_MAX - 4096;

inline bool shapes_fit(int batch, int dim, int64_t seqlen) {
  if (batch < 0 || dim < 0 || seqlen < 0 || seqlen > kMaxSeqlen) return false;
  const long double total = (long double)batch * (long double)dim * (long double)(seqlen > 0 ? seqlen : 1);
  return total < (long double)(INT64_C(1) << 60);
}

}  // namespace ssm
