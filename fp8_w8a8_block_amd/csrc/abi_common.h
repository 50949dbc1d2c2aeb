// What the files of the C ABI share: bounds on shapes, byte ranges, the device
// check and the status of a launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstring>

#include "fp8w8a8.h"

namespace fp8abi {

constexpr int64_t kMaxDim = (int64_t)1 << 31;        // any single extent
constexpr int64_t kMaxElems = (int64_t)1 << 40;      // rows * cols of one tensor
constexpr int64_t kMaxSpan = (int64_t)1 << 56;       // rows * ld of one tensor (elements)

// rows rows at leading dimension ld span at most kMaxSpan elements, so every
// byte range below is computed without overflow
inline bool span_ok(int64_t rows, int64_t ld) {
  return ld >= 0 && ld <= kMaxSpan && (rows <= 1 || ld <= kMaxSpan / rows);
}

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Byte range [lo, hi) of a row-major matrix.
struct Range {
  uintptr_t lo, hi;
};
inline Range range_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  uintptr_t lo = (uintptr_t)p;
  if (rows <= 0 || cols <= 0) return {lo, lo};
  uintptr_t hi = lo + (uintptr_t)(((rows - 1) * ld + cols) * elem);
  return {lo, hi};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Per-device cache of "is this a gfx950": 0 unknown, 1 yes, 2 no.
constexpr int kMaxDevices = 64;
inline std::atomic<int> g_arch_ok[kMaxDevices];

inline fp8_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return FP8_ERR_DEVICE;
  int state = g_arch_ok[dev].load(std::memory_order_relaxed);
  if (state == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return FP8_ERR_DEVICE;
    state = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_arch_ok[dev].store(state, std::memory_order_relaxed);
  }
  return state == 1 ? FP8_OK : FP8_ERR_DEVICE;
}

inline fp8_status launched(hipError_t e) { return e == hipSuccess ? FP8_OK : FP8_ERR_LAUNCH; }

}  // namespace fp8abi
