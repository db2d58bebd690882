// Rows in the registers of a few wavefronts: what the layer norm (norm_kernels.hip) and
// root-mean-square norm (rms_kernels.hip) kernels share. Sums over the lanes and wavefronts of a
// row, the columns that a lane owns, the launch shapes by row length and the reduction of the
// workgroups' partial parameter gradients.
#pragma once

#include <algorithm>

#include "common.h"
#include "elem.h"

namespace lce {
namespace {

// Sum over a wavefront, the same bits in every lane. The steps within 16 lanes are data-parallel
// moves of the VALU and the last two exchange rows of lanes between two registers, so none goes
// through the LDS permute that a shuffle is: the sums of a row are on its critical path.
template <int CTRL>
__device__ __forceinline__ float add_lanes(float x) {
  const int y = __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true);
  return x + __int_as_float(y);
}
__device__ __forceinline__ float wave_sum(float x) {
  x = add_lanes<0xB1>(x);   // lane ^ 1
  x = add_lanes<0x4E>(x);   // lane ^ 2
  x = add_lanes<0x141>(x);  // mirrored within 8: the other four
  x = add_lanes<0x140>(x);  // mirrored within 16: the other eight
  int i = __float_as_int(x);
  const auto r = __builtin_amdgcn_permlane16_swap(i, i, false, false);
  i = __float_as_int(__int_as_float(r[0]) + __int_as_float(r[1]));
  const auto h = __builtin_amdgcn_permlane32_swap(i, i, false, false);
  return __int_as_float(h[0]) + __int_as_float(h[1]);
}

// Threads of a workgroup for rows of WPR wavefronts: several rows side by side where few
// wavefronts hold one.
constexpr int norm_threads(int wpr, int least) { return 64 * wpr > least ? 64 * wpr : least; }

// The sums of K values over the WPR wavefronts that share a row, in wavefront order. `red` is
// used for one reduction at a time: the caller alternates two of them, so that a wavefront that
// runs ahead into the next reduction does not overwrite values still being read.
template <int WPR, int K>
__device__ __forceinline__ void row_sums(float (&x)[K], float (*red)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = wave_sum(x[k]);
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[wave][k] = x[k];
    }
    __syncthreads();
    const int w0 = wave / WPR * WPR;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k] = red[w0][k];
#pragma unroll
      for (int w = 1; w < WPR; ++w) x[k] += red[w0 + w][k];
    }
  }
}

// The vectors a lane owns of a row of h elements: vector j starts at column at[j], and its
// elements from skip[j] on are the lane's to count (none where the vector lies past the row).
// Where h is no multiple of the vector, the row's last vector is moved back to end with the row
// and skips what the one before it holds (both lanes compute and store the same values there), so
// that every access is a whole vector; a vector past the row reads the row's first and is not
// stored. FULL: h is a multiple of the vector, a vector counts wholly or not at all.
template <int VE, int NV, int LANES, bool FULL>
struct Columns {
  int h, at[NV], skip[NV];
  __device__ __forceinline__ Columns(int lane, int h_) : h(h_) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (lane + j * LANES) * VE;
      at[j] = c >= h ? 0 : c + VE <= h ? c : h < VE ? 0 : h - VE;
      skip[j] = c >= h ? VE : c - at[j];
    }
  }
  __device__ __forceinline__ bool live(int j) const { return skip[j] < VE; }
  __device__ __forceinline__ bool counts(int j, int q) const {
    return FULL ? skip[j] == 0 : q >= skip[j] && q < h;
  }
  template <bool STREAM = false, class T>
  __device__ __forceinline__ raw4 load(const T* row, int j) const {
    if (!FULL && h < VE) {  // a row shorter than a vector, uniformly
      float x[VE];
#pragma unroll
      for (int q = 0; q < VE; ++q) x[q] = q < h ? Elem<T>::to_f32(row[q]) : 0.f;
      return Elem<T>::pack(x);
    }
    return STREAM ? load_stream(row + at[j]) : load_raw(row + at[j]);
  }
  template <bool STREAM = false, class T>
  __device__ __forceinline__ void store(T* row, int j, const float (&x)[VE]) const {
    if (!FULL && h < VE) {
#pragma unroll
      for (int q = 0; q < VE; ++q)
        if (q < h) row[q] = Elem<T>::from_f32(x[q]);
    } else {
      if (STREAM)
        store_stream(row + at[j], Elem<T>::pack(x));
      else
        store_raw(row + at[j], Elem<T>::pack(x));
    }
  }
  // A parameter at the lane's columns, `none` where there is none.
  template <class P>
  __device__ __forceinline__ void param(const P* p, int j, float none, float (&x)[VE]) const {
    if (p) {
      load_some<P, VE>(p + at[j], !FULL && h < VE ? h : VE, x);
    } else {
#pragma unroll
      for (int q = 0; q < VE; ++q) x[q] = none;
    }
  }
};

// dw and db from the workgroups' partial rows: 32 columns per workgroup, the rows dealt to
// eight thread groups, their sums added in group order. blockIdx.y: 0 weight, 1 bias.
constexpr int kRedCols = 32, kRedGroups = 8;
template <class P, bool ACC>
__global__ void __launch_bounds__(kRedCols* kRedGroups) param_reduce_kernel(
    const float* __restrict__ part_w, const float* __restrict__ part_b, int64_t rows, int64_t h,
    P* dw, P* db) {
  P* out = blockIdx.y ? db : dw;
  if (!out) return;
  const float* part = blockIdx.y ? part_b : part_w;
  __shared__ float sum[kRedGroups][kRedCols];
  const int lane = threadIdx.x % kRedCols, q = threadIdx.x / kRedCols;
  const int64_t c = int64_t(blockIdx.x) * kRedCols + lane;
  float s = 0.f;
  if (c < h) {
#pragma unroll 8
    for (int64_t r = q; r < rows; r += kRedGroups) s += part[r * h + c];
  }
  sum[q][lane] = s;
  __syncthreads();
  if (q == 0 && c < h) {
    float t = sum[0][lane];
#pragma unroll
    for (int k = 1; k < kRedGroups; ++k) t += sum[k][lane];
    if (ACC) t += Elem<P>::to_f32(out[c]);
    out[c] = Elem<P>::from_f32(t);
  }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Calls f with the row shape (WPR, EPL) for rows of h elements: up to E elements a lane, fewer
// where one wavefront holds the row with fewer; wavefronts per row doubled until the row fits.
// For E = 16, rows that leave a quarter or more of the next shape empty take half the wavefronts
// with 24 elements a lane, and eight wavefronts hold up to 32, since sixteen have half the registers
// each and spill ([3000, 10001] fp16 71 us so and 123 on sixteen, [2048, 16384] bf16 56 and 73). Rows
// past that take sixteen with 32.
template <int E, class F>
hipError_t with_shape(int64_t h, F&& f) {
  using std::integral_constant;
  using W1 = integral_constant<int, 1>;
  using W2 = integral_constant<int, 2>;
  using W4 = integral_constant<int, 4>;
  using W8 = integral_constant<int, 8>;
  using W16 = integral_constant<int, 16>;
  using EE = integral_constant<int, E>;
  using E24 = integral_constant<int, 24>;
  using E32 = integral_constant<int, 32>;
  if (h <= 512) return f(W1{}, integral_constant<int, 8>{});
  if (h <= 1024) return f(W1{}, integral_constant<int, 16>{});
  if constexpr (E == 16) {
    if (h <= 64 * 24) return f(W1{}, E24{});
    if (h <= 128 * 16) return f(W2{}, EE{});
    if (h <= 128 * 24) return f(W2{}, E24{});
    if (h <= 256 * 16) return f(W4{}, EE{});
    if (h <= 256 * 24) return f(W4{}, E24{});
    if (h <= 512 * 16) return f(W8{}, EE{});
    if (h <= 512 * 24) return f(W8{}, E24{});
    if (h <= 512 * 32) return f(W8{}, E32{});
  } else {
    static_assert(E == 32, "E");
    if (h <= 64 * 32) return f(W1{}, E32{});
    if (h <= 128 * 32) return f(W2{}, E32{});
    if (h <= 256 * 32) return f(W4{}, E32{});
    if (h <= 512 * 32) return f(W8{}, E32{});
  }
  return f(W16{}, E32{});
}

template <class P>
hipError_t run_reduce(const float* pw, const float* pb, int64_t rows, int64_t h, bool add, void* dw,
                      void* db, hipStream_t s) {
  const dim3 grid(unsigned((h + kRedCols - 1) / kRedCols), db ? 2 : 1);
  TimedLaunch t(s, K_NORM_PARAM_REDUCE);
  if (add)
    hipLaunchKernelGGL((param_reduce_kernel<P, true>), grid, dim3(kRedCols * kRedGroups), 0, s, pw,
                       pb, rows, h, static_cast<P*>(dw), static_cast<P*>(db));
  else
    hipLaunchKernelGGL((param_reduce_kernel<P, false>), grid, dim3(kRedCols * kRedGroups), 0, s,
                       pw, pb, rows, h, static_cast<P*>(dw), static_cast<P*>(db));
  return hipGetLastError();
}

}  // namespace
}  // namespace lce
