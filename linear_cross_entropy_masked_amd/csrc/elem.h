// Element types of the embedding and layer norm kernels (bf16, fp16, fp32) and their vector
// accesses: sixteen bytes per lane at element alignment. Rows of any stride and width therefore
// take the same path (global memory accesses may be unaligned on gfx950: the compiler emits one
// 16-byte instruction for these), and only a row's last, partial vector goes element by element.
#pragma once

#include "common.h"

namespace lce {

enum Dtype { kBF16 = 0, kF16 = 1, kF32 = 2 };  // LCE_DTYPE_* of the C ABI

struct Bf16 {
  uint16_t bits;
};

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t raw4_b2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t raw4_b4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t raw4 __attribute__((ext_vector_type(4)));

template <class T>
struct Elem;

template <>
struct Elem<Bf16> {
  static constexpr int kVec = 8;  // elements of a 16-byte vector
  using Raw = raw4_b2;
  static __device__ __forceinline__ float to_f32(Bf16 x) { return bf16_to_f32(x.bits); }
  static __device__ __forceinline__ Bf16 from_f32(float x) { return Bf16{f32_to_bf16(x)}; }
  static __device__ __forceinline__ void unpack(raw4 r, float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = bf16_lo(r[k]);
      x[2 * k + 1] = bf16_hi(r[k]);
    }
  }
  static __device__ __forceinline__ raw4 pack(const float (&x)[8]) {
    return raw4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                pack_bf16x2(x[6], x[7])};
  }
};

template <>
struct Elem<_Float16> {
  static constexpr int kVec = 8;
  using Raw = raw4_b2;
  static __device__ __forceinline__ float to_f32(_Float16 x) { return float(x); }
  static __device__ __forceinline__ _Float16 from_f32(float x) { return _Float16(x); }
  static __device__ __forceinline__ void unpack(raw4 r, float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f16x2_t p = __builtin_bit_cast(f16x2_t, uint32_t(r[k]));
      x[2 * k] = float(p.x);
      x[2 * k + 1] = float(p.y);
    }
  }
  static __device__ __forceinline__ raw4 pack(const float (&x)[8]) {
    raw4 r;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      r[k] = __builtin_bit_cast(uint32_t, f16x2_t{_Float16(x[2 * k]), _Float16(x[2 * k + 1])});
    return r;
  }
};

template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  using Raw = raw4_b4;
  static __device__ __forceinline__ float to_f32(float x) { return x; }
  static __device__ __forceinline__ float from_f32(float x) { return x; }
  static __device__ __forceinline__ void unpack(raw4 r, float (&x)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(r[k]);
  }
  static __device__ __forceinline__ raw4 pack(const float (&x)[4]) {
    return raw4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                __float_as_uint(x[3])};
  }
};

template <class T>
__device__ __forceinline__ raw4 load_raw(const T* p) {
  return *reinterpret_cast<const typename Elem<T>::Raw*>(p);
}
template <class T>
__device__ __forceinline__ void store_raw(T* p, raw4 r) {
  *reinterpret_cast<typename Elem<T>::Raw*>(p) = r;
}

// The same for rows that are read or written once (non-temporal).
template <class T>
__device__ __forceinline__ raw4 load_stream(const T* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const typename Elem<T>::Raw*>(p));
}
template <class T>
__device__ __forceinline__ void store_stream(T* p, raw4 r) {
  __builtin_nontemporal_store(static_cast<typename Elem<T>::Raw>(r),
                              reinterpret_cast<typename Elem<T>::Raw*>(p));
}

// `cnt` elements at p into x (the others 0); cnt >= N: one vector access.
template <class T, int N>
__device__ __forceinline__ void load_some(const T* p, int64_t cnt, float (&x)[N]) {
  if (cnt >= N) {
    if constexpr (N == Elem<T>::kVec) {
      Elem<T>::unpack(load_raw(p), x);
    } else {  // fp32 beside a 16-bit type: two vectors
      static_assert(N == 2 * Elem<T>::kVec, "N");
      float a[Elem<T>::kVec], b[Elem<T>::kVec];
      Elem<T>::unpack(load_raw(p), a);
      Elem<T>::unpack(load_raw(p + Elem<T>::kVec), b);
#pragma unroll
      for (int k = 0; k < Elem<T>::kVec; ++k) {
        x[k] = a[k];
        x[Elem<T>::kVec + k] = b[k];
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = k < cnt ? Elem<T>::to_f32(p[k]) : 0.f;
  }
}
template <class T, int N>
__device__ __forceinline__ void store_some(T* p, int64_t cnt, const float (&x)[N]) {
  if (cnt >= N) {
    if constexpr (N == Elem<T>::kVec) {
      store_raw(p, Elem<T>::pack(x));
    } else {
      static_assert(N == 2 * Elem<T>::kVec, "N");
      float a[Elem<T>::kVec], b[Elem<T>::kVec];
#pragma unroll
      for (int k = 0; k < Elem<T>::kVec; ++k) {
        a[k] = x[k];
        b[k] = x[Elem<T>::kVec + k];
      }
      store_raw(p, Elem<T>::pack(a));
      store_raw(p + Elem<T>::kVec, Elem<T>::pack(b));
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < cnt) p[k] = Elem<T>::from_f32(x[k]);
  }
}

}  // namespace lce
