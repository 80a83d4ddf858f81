// rows.h — checks of pointers and rows that a caller of the C ABI passes (host
// code).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/h2o.h"

namespace h2o {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Reads of a row start at 16-byte boundaries; `step`: elements in 16 bytes.
inline bool rows_fit(const h2o_rows *r, int step) {
  if (!r || !r->data || !aligned(r->data, 16)) return false;
  return r->stride_b >= 0 && r->stride_h >= 0 && r->stride_t >= 0 && r->stride_b % step == 0 &&
         r->stride_h % step == 0 && r->stride_t % step == 0;
}
// No two rows of an output share memory: in the order of their strides, each
// dimension steps over everything the smaller ones span.
inline bool rows_apart(const h2o_rows *r, int B, int H, int n, int d) {
  int64_t size[3] = {B, H, n}, step[3] = {r->stride_b, r->stride_h, r->stride_t};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (step[j] < step[i]) {
        const int64_t s = step[i], z = size[i];
        step[i] = step[j], size[i] = size[j];
        step[j] = s, size[j] = z;
      }
  int64_t span = d;
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;
    if (step[i] < span) return false;
    span = step[i] * (size[i] - 1) + span;
  }
  return true;
}

}  // namespace h2o
