// Internal interface of the decoding operators (rope.cu, cache.cu, tree.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pbs.h"

namespace pbs {

// The device error word of the current device (api.cu).
int *error_word();

// 16-byte aligned rows: base and every used stride.
inline bool rows_ok(const pbs_rows &r, int elem) {
  const int64_t v = 16 / elem;
  return r.p && ((uintptr_t)r.p & 15u) == 0 && r.layer % v == 0 && r.batch % v == 0 &&
         r.head % v == 0 && r.row % v == 0;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace pbs
