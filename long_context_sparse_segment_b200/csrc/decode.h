// Internal interface of the decoding operators (rope.cu, cache.cu, tree.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

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

// Whether [a, a + an) and [b, b + bn) meet; a null one meets nothing.
inline bool bytes_meet(const void *a, int64_t an, const void *b, int64_t bn) {
  return a && b && an > 0 && bn > 0 && (uintptr_t)a < (uintptr_t)b + (uintptr_t)bn &&
         (uintptr_t)b < (uintptr_t)a + (uintptr_t)an;
}

// Rows [batch, heads, n, d] of `elem` bytes an element.
struct RowSet {
  pbs_rows r;
  int64_t batch, heads, n;
  int d, elem;
  // the bytes from the lowest element, and how many up to behind the highest
  const uint8_t *low() const { return (const uint8_t *)r.p + elem * reach(-1); }
  int64_t bytes() const { return elem * (reach(1) - reach(-1) + d); }
  bool plain() const { return reach(-1) == 0; }  // no stride runs backwards
  bool empty() const { return batch <= 0 || heads <= 0 || n <= 0 || d <= 0; }

 private:
  int64_t reach(int sign) const {  // elements from p to the last row that way
    auto part = [&](int64_t stride, int64_t size) {
      return stride * sign > 0 ? stride * (size - 1) : 0;
    };
    return part(r.batch, batch) + part(r.head, heads) + part(r.row, n);
  }
};

// Whether two sets of rows share memory: element by element where their strides
// are equal (slices of one buffer, which may interleave), else by their spans.
bool rows_meet(const RowSet &x, const RowSet &y);
// ... and whether a set of rows and some bytes do, by the span.
bool rows_meet(const RowSet &x, const void *p, int64_t bytes);

// SMs of the current device, looked up once per device.
int sm_count_cached();

// The dynamic shared memory of a kernel allowed once per device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit & done.load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace pbs
