// row_slices.hpp -- batch rows over the second dimension of several launches.
#pragma once

#include <cstdint>

namespace ssm {

constexpr int kMaxGridRows = 65535;  // of one launch

// f(first row, rows) for one slice of the batch after another, until a result is
// not `ok`; that result, or `ok`.  The position is held in 64 bits: behind the last
// of nearly 2^31 rows it is past 32.
template <typename R, typename F>
R by_row_slices(int batch, R ok, F&& f) {
  for (int64_t b0 = 0; b0 < batch; b0 += kMaxGridRows) {
    const int64_t left = batch - b0;
    const R r = f((int)b0, (int)(left < kMaxGridRows ? left : kMaxGridRows));
    if (r != ok) return r;
  }
  return ok;
}

}  // namespace ssm
