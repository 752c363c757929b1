// Host helpers of the C ABI's argument checks and launches.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "row_overlap.h"

namespace moe {

// The calling thread's device, set for a scope (and left alone where it is the one already).
struct Device {
  int prev = -1;
  bool ok = false;
  explicit Device(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    ok = prev == dev || cudaSetDevice(dev) == cudaSuccess;
    if (prev == dev) prev = -1;
  }
  ~Device() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// A bf16 array of rows of `width` values, `stride` apart.
inline bool rows_ok(const void* p, int64_t stride, int64_t width) {
  return p && aligned16(p) && stride >= width && stride % 8 == 0;
}

// Whether two arrays of rows (row stride and width in bf16 values) share a byte.
inline bool overlap_rows(const void* a, int64_t as, int64_t aw, const void* b, int64_t bs,
                         int64_t bw, int rows) {
  return rows_overlap(reinterpret_cast<uintptr_t>(a), 2 * as, 2 * aw,
                      reinterpret_cast<uintptr_t>(b), 2 * bs, 2 * bw, rows);
}

// The driver's tensor map encoder, or nullptr where there is no driver.
inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    cudaGetLastError();
  });
  return fn;
}

}  // namespace moe
