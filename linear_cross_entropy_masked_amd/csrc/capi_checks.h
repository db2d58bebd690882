// Argument checks shared by the C-ABI entry points: sizes, alignment, the device, and which byte
// ranges of a call may meet.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstring>
#include <limits>

#include "lce_masked.h"

namespace lce {
namespace {

constexpr int64_t kI64Max = std::numeric_limits<int64_t>::max();

bool mul_overflows(int64_t a, int64_t b) { return a != 0 && b > kI64Max / a; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Per-device cache: 0 = unknown, 1 = gfx950, 2 = other.
std::atomic<int> g_arch_ok[64];

int check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return LCE_ERR_HIP;
  if (dev >= 0 && dev < 64) {
    int c = g_arch_ok[dev].load(std::memory_order_relaxed);
    if (c) return c == 1 ? LCE_OK : LCE_ERR_DEVICE;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return LCE_ERR_HIP;
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev >= 0 && dev < 64) g_arch_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? LCE_OK : LCE_ERR_DEVICE;
}

// Byte range [lo, hi) a call reads or writes; empty for a NULL pointer or no bytes.
struct Span {
  uintptr_t lo, hi;
};
Span span(const void* p, int64_t bytes) {
  if (!p || bytes <= 0) return Span{0, 0};
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + uintptr_t(bytes)};
}
// Bytes of a row-major [n, ld] matrix whose first `cols` columns are used.
int64_t matrix_bytes(int64_t n, int64_t ld, int64_t cols, int64_t elem) {
  return n > 0 ? ((n - 1) * ld + cols) * elem : 0;
}
bool spans_meet(Span a, Span b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}
// Every written range must be disjoint from every read range and from the other written
// ranges (inputs may share memory with each other).
template <size_t NW, size_t NR>
int check_disjoint(const Span (&wr)[NW], const Span (&rd)[NR]) {
  for (size_t i = 0; i < NW; ++i) {
    for (size_t j = 0; j < NR; ++j)
      if (spans_meet(wr[i], rd[j])) return LCE_ERR_OVERLAP;
    for (size_t j = i + 1; j < NW; ++j)
      if (spans_meet(wr[i], wr[j])) return LCE_ERR_OVERLAP;
  }
  return LCE_OK;
}

#define LCE_TRY_HIP(expr)                        \
  do {                                           \
    if ((expr) != hipSuccess) return LCE_ERR_HIP; \
  } while (0)

}  // namespace
}  // namespace lce
