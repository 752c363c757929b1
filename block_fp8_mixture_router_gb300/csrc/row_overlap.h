// Whether two arrays of rows share memory, for the host: plain C++, no CUDA.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {

// Whether `rows` rows of bytes at a (aw bytes every as) and at b (bw every bs) share a
// byte; 0 < aw <= as, 0 < bw <= bs, rows >= 1.  Column ranges of one buffer lie between one
// another and share none.
inline bool rows_overlap(uintptr_t a, int64_t as, int64_t aw, uintptr_t b, int64_t bs, int64_t bw,
                         int64_t rows) {
  const int64_t last = rows - 1;
  const int64_t d = (int64_t)(b - a);  // of two addresses of one space: fits
  if (d >= as * last + aw || -d >= bs * last + bw) return false;  // one behind the other
  // The last row j of b that begins before row i of a ends, if it ends behind row i's
  // beginning: d + j bs < i as + aw and d + j bs + bw > i as.
  const auto floor_div = [](int64_t x, int64_t y) { return x >= 0 ? x / y : -((y - 1 - x) / y); };
  if (as == bs) {  // the same for all i: by k = j - i
    const int64_t k = std::min(floor_div(aw - 1 - d, bs), last);
    return k >= -last && d + k * bs + bw > 0;
  }
  for (int64_t i = 0; i <= last; ++i) {
    const int64_t j = std::min(floor_div(i * as + aw - 1 - d, bs), last);
    if (j >= 0 && d + j * bs + bw > i * as) return true;
  }
  return false;
}

}  // namespace moe
