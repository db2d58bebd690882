// 8-bit floating point (e4m3: 1 sign, 4 exponent, 3 mantissa bits, largest 448) in blocks of 128
// columns that share a scale.
//
//   a = max |y| over the block,  c = max(a / 448, 2^-126),  q = e4m3(y / c)
//
// c is held in fp32, or rounded up to a power of two and held as its exponent byte (e8m0: 2^(byte
// - 127)). |y / c| stays within 448 (1 + 2^-23), which rounds to 448, so nothing is clamped. A
// block that holds a NaN or an infinity gets the scale NaN (byte 255) and NaN values throughout.
#pragma once

#include "common.h"
#include "elem.h"

namespace lce {

enum ScaleType { kScaleF32 = 0, kScaleE8M0 = 1 };  // LCE_SCALE_* of the C ABI

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.f;
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kNanBits = 0x7fc00000u;
constexpr uint32_t kOneBits = 0x3f800000u;

// |x| as an integer that orders like the number, NaN above infinity: the largest of a block then
// keeps a NaN, which a floating-point maximum drops.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The scale of a block from abs_bits() of its largest element: what is stored, and its reciprocal
// (exact for a power of two). An element is divided by an fp32 scale by Markstein's correction (1990):
// from the rounded reciprocal, one step with the exact remainder rounds the quotient correctly, in
// three operations where a general division takes ten (2048 x 4096 bf16 in 6.9 us and 8.5).
template <bool POW2>
struct BlockScale {
  uint32_t held;
  float c, inv;
  __device__ __forceinline__ explicit BlockScale(uint32_t largest) {
    c = fmaxf(__uint_as_float(largest) / kFp8Max, 0x1p-126f);
    const bool bad = largest >= kInfBits;
    if (POW2) {
      // any mantissa bit carries into the exponent; c is normal and far below 2^127
      const uint32_t e = bad ? 255u : (__float_as_uint(c) + 0x7fffffu) >> 23;
      held = e;
      inv = __uint_as_float(bad ? kNanBits : (254u - e) << 23);
    } else {
      held = bad ? kNanBits : __float_as_uint(c);
      c = __uint_as_float(held);
      inv = 1.f / c;
    }
  }
  __device__ __forceinline__ float scaled(float y) const {
    const float q = y * inv;
    return POW2 ? q : fmaf(fmaf(-q, c, y), inv, q);
  }
  __device__ __forceinline__ void store(void* scales, int64_t at) const {
    if (POW2)
      static_cast<uint8_t*>(scales)[at] = uint8_t(held);
    else
      static_cast<uint32_t*>(scales)[at] = held;
  }
};

// Four values in 8 bits each, to nearest even.
__device__ __forceinline__ uint32_t pack_fp8x4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

typedef uint32_t raw1_b1 __attribute__((aligned(1)));
typedef uint32_t raw2 __attribute__((ext_vector_type(2)));
typedef uint32_t raw2_b1 __attribute__((ext_vector_type(2), aligned(1)));

// The elements [skip, end) of N (4 or 8) scaled values at p, in one access where that is all.
template <bool POW2, int N>
__device__ __forceinline__ void store_fp8(uint8_t* p, const BlockScale<POW2>& s,
                                          const float (&y)[N], int skip, int end) {
  static_assert(N == 4 || N == 8, "N");
  uint32_t w[N / 4];
#pragma unroll
  for (int k = 0; k < N / 4; ++k)
    w[k] = pack_fp8x4(s.scaled(y[4 * k]), s.scaled(y[4 * k + 1]), s.scaled(y[4 * k + 2]),
                      s.scaled(y[4 * k + 3]));
  if (skip == 0 && end >= N) {
    if constexpr (N == 8)
      *reinterpret_cast<raw2_b1*>(p) = raw2{w[0], w[1]};
    else
      *reinterpret_cast<raw1_b1*>(p) = w[0];
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k >= skip && k < end) p[k] = uint8_t(w[k / 4] >> (8 * (k % 4)));
  }
}

// The largest of 16 (32 for WIDE) neighbouring lanes, in all of them.
template <int CTRL>
__device__ __forceinline__ uint32_t max_lanes(uint32_t x) {
  const uint32_t y = uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CTRL, 0xf, 0xf, true));
  return x > y ? x : y;
}
template <bool WIDE>
__device__ __forceinline__ uint32_t max_of_16(uint32_t x) {
  x = max_lanes<0xB1>(x);   // lane ^ 1
  x = max_lanes<0x4E>(x);   // lane ^ 2
  x = max_lanes<0x141>(x);  // mirrored within 8
  x = max_lanes<0x140>(x);  // mirrored within 16
  if (WIDE) {
    const auto r = __builtin_amdgcn_permlane16_swap(int(x), int(x), false, false);
    x = uint32_t(r[0]) > uint32_t(r[1]) ? uint32_t(r[0]) : uint32_t(r[1]);
  }
  return x;
}

}  // namespace lce
