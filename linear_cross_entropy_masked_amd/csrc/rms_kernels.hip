// Root-mean-square norm of a sum, forward (16- / 32-bit or 8-bit outputs) and backward for gfx950.
//
//   forward   s = x + residual, rounded to their type;  r = 1 / sqrt(mean(s²) + eps) per row
//             y = s · r · w, or y in 8 bits with a scale for each block of 128 columns (fp8.h)
//   backward  u = g · w,  ŝ = s · r
//             ds = r · (u − ŝ · mean(u · ŝ)) + g_s          per row, g_s the gradient of s itself
//             dw (=|+=) Σ_rows g · ŝ
//
// The norm is that of the rounded s: s is what the model carries on, and what the backward reads.
// Memory-bound, as layer norm (norm_kernels.hip), and built like it: a row lives in the registers
// of WPR wavefronts from its one read to its one write, the next row is loaded before the sums of
// this, and dw goes through one partial row per workgroup, added in workgroup order. A block of 128
// columns is 16 (fp32: 32) neighbouring lanes' vectors, so its largest element takes four or five
// lane exchanges and no LDS.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "elem.h"
#include "fp8.h"
#include "norm_rows.h"
#include "ops.h"

namespace lce {

namespace {

// Launch shapes, with x + residual read, their sum and a 16-bit (8-bit) y written, in us:
//                                        [65536, 4096] bf16   [4096, 4096] bf16   [20001, 1025] fp16
//   512 threads, 16 elements a lane         367  (300)            21.9 (21.9)         36.9 (45.1)
//   512 threads, 32 elements                377  (340)            26.8 (27.0)         47.8 (53.4)
//   256 threads, 16 elements                402  (311)            22.1 (22.5)         37.3 (40.8)
//   256 threads, 32 elements                372  (301)            23.0 (23.8)         45.3 (48.8)
// 367 us are 5.9 TB/s (a large copy: 4.9). The grid is what 2048 workgroups of 512 threads hold;
// half or twice of that makes 362 and 408 us, 22.9 and 21.8. The backward ([8192, 4096] bf16 with
// the gradient of the sum, 5.1 TB/s, and [4099, 2051] fp16): 256 threads and 512 workgroups 49.5
// and 18.6 us, 513 workgroups 53.6 and 23.0, 768 50.1 and 20.0, 1024 58.5 and 20.2; held as loaded
// and widened for each use as long rows are, 54.1 and 20.4. Adding the partial rows takes 4.5 us
// of both.
constexpr int kFwdThreads = 512, kFwdElems = 16;
constexpr int kBwdThreads = 256, kBwdElems = 16;
constexpr int64_t kFwdGrid = 2048;
constexpr int64_t kShortRow = 512, kPairRow = 256 * 24, kRegRow = 512 * 32;
constexpr int64_t kColRows = 64, kLongGrid = 512;
// Of fp32 rows, half as many numbers with their dw fit a workgroup's registers ([1538, 12728] fp32
// with the gradient of the sum: 104 us as long rows, 138 else).
template <class T>
constexpr int64_t kRegRowOf = sizeof(T) == 4 ? kRegRow / 2 : kRegRow;
int64_t bwd_grid(int64_t h) { return h <= kShortRow ? 1024 : h <= kPairRow ? 512 : 256; }
template <class T>
int64_t part_rows(int64_t n, int64_t h) {
  return std::min(n, h > kRegRowOf<T> ? kColRows : bwd_grid(h));
}
// A forward of whole vectors that moves more than this passes by the caches (non-temporal loads and
// stores): 512 MiB take 92 us so and 111 without, 128 MiB 22 either way, 64 MiB 17.4 and 16.3.
constexpr int64_t kStreamBytes = int64_t(256) << 20;

// A weight of the rows' own type or of fp32, at a lane's columns.
template <class T, class C, int VE>
__device__ __forceinline__ void weight_at(const C& col, const void* w, bool wide, int j,
                                          float (&x)[VE]) {
  if (wide)
    col.param(static_cast<const float*>(w), j, 1.f, x);
  else
    col.param(static_cast<const T*>(w), j, 1.f, x);
}

// The weight at a lane's columns: held from the start (HOLD), so that no row waits for it behind its
// sums, or loaded where a row needs it, in a forward of sixteen wavefronts a row, which has no
// registers to spare, and in one to 16 bits that passes by the caches, where the wavefronts that
// the registers cost matter more. Held and not: to 8 bits [8192, 8192] bf16 76.5 and 82.0 us, [65536,
// 4096] 292 and 300; 16 bits [20001, 1025] fp16 34.9 and 36.8, [65536, 4096] 388 and 366; backward
// [8192, 4096] bf16 52.9 and 55.3, [4099, 2051] fp16 18.3 and 21.3, [20001, 1025] 40.0 and 48.5.
template <class T, class C, int VE, int NV, bool HOLD>
struct Weight {
  const void* p;
  bool wide;
  float held[HOLD ? NV : 1][VE];
  __device__ __forceinline__ Weight(const C& col, const void* p_, bool wide_) : p(p_), wide(wide_) {
    if constexpr (HOLD) {
#pragma unroll
      for (int j = 0; j < NV; ++j) weight_at<T>(col, p, wide, j, held[j]);
    }
  }
  __device__ __forceinline__ void get(const C& col, int j, float (&x)[VE]) const {
    if constexpr (HOLD) {
#pragma unroll
      for (int q = 0; q < VE; ++q) x[q] = held[j][q];
    } else {
      weight_at<T>(col, p, wide, j, x);
    }
  }
};

struct RmsFwd {
  const void *x, *residual, *weight;
  int64_t n, ldx, ldr;
  int h;
  bool wide;  // an fp32 weight
  float eps;
  void *y, *sum;  // y: rows of x's type, or 8-bit ones
  int64_t ldy, ldsum;
  float* rstd;
  void* scales;  // 8-bit outputs
  int64_t lds;
  bool pow2;
};

// The wavefront's sum in all lanes; no step goes through LDS.
__device__ __forceinline__ double wave_add_f64(double x) {
  auto lanes = [&](auto ctrl) {
    constexpr int CTRL = decltype(ctrl)::value;
    const uint64_t u = __double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(u), CTRL, 0xf, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(u >> 32), CTRL, 0xf, 0xf, true);
    x += __longlong_as_double(uint64_t(hi) << 32 | lo);
  };
  lanes(std::integral_constant<int, 0xB1>{});   // lane ^ 1
  lanes(std::integral_constant<int, 0x4E>{});   // lane ^ 2
  lanes(std::integral_constant<int, 0x141>{});  // mirrored within 8
  lanes(std::integral_constant<int, 0x140>{});  // mirrored within 16
  auto halves = [&](auto swap) {
    const uint64_t u = __double_as_longlong(x);
    const auto lo = swap(int(u)), hi = swap(int(u >> 32));
    x = __longlong_as_double(uint64_t(uint32_t(hi[0])) << 32 | uint32_t(lo[0])) +
        __longlong_as_double(uint64_t(uint32_t(hi[1])) << 32 | uint32_t(lo[1]));
  };
  halves([](int v) { return __builtin_amdgcn_permlane16_swap(v, v, false, false); });
  halves([](int v) { return __builtin_amdgcn_permlane32_swap(v, v, false, false); });
  return x;
}

// The sum over the WPR wavefronts that share a row, in wavefront order; `red` as for row_sums().
// In fp64 from the lanes' fp32 sums on, so that what it is off by is their few roundings averaged
// over all lanes.
template <int WPR>
__device__ __forceinline__ double row_sum_f64(double x, double* red) {
  x = wave_add_f64(x);
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = x;
    __syncthreads();
    const int w0 = wave / WPR * WPR;
    x = red[w0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) x += red[w0 + w];
  }
  return x;
}

// 1 / sqrt(mean + eps) in two parts, and v times it times w rounded once.
struct Rstd {
  double exact;
  float hi, lo;
  __device__ __forceinline__ Rstd(double sum, const RmsFwd& a)
      : exact(1.0 / sqrt(sum / a.h + a.eps)), hi(float(exact)), lo(float(exact - hi)) {}
  __device__ __forceinline__ float times(float v, float w) const {
    const float p = v * hi;
    if (!(hi < INFINITY)) return p * w;  // eps and all of the row 0
    return fmaf(p, w, fmaf(v, lo, fmaf(v, hi, -p)) * w);
  }
  // The same for a weight that may be infinite, beside which what p is off by would count as 0 · inf
  // or inf - inf: kept finite (a NaN among the three becomes the least), which a finite weight's is.
  // A block of 8 bits is NaN throughout either way. A branch on the weight instead cost [20001, 1025]
  // fp32 71.0 us, 66.5 without it.
  __device__ __forceinline__ float times_any(float v, float w) const {
    const float p = v * hi;
    if (!(hi < INFINITY)) return p * w;
    const float off = fmaf(v, lo, fmaf(v, hi, -p)) * w;
    return fmaf(p, w, __builtin_amdgcn_fmed3f(off, -__FLT_MAX__, __FLT_MAX__));
  }
};

// A row's sums v as y = v · rstd · weight in 8 bits. With rstd in two parts and what the product
// with v is off by carried along, y is the real number rounded once to fp32, so that no second
// rounding moves it past a tie of the 8-bit numbers (one in 200 000). A block whose largest y then
// lies beside 448 · 2^k, where a scale that is a power of two doubles, has it formed in fp64. The
// registers of that, kept to 128 by the launch bounds, cost rows of 24 elements a lane a tenth
// ([3000, 6000] bf16 30.0 us, 27.4 without), those of 16 nothing.
template <bool POW2, class T, int VE, int NV, class C, class W>
__device__ __forceinline__ void store_row_fp8(const C& col, const RmsFwd& a, int64_t r, int lane,
                                              int stride, const float (&v)[NV][VE], const W& weight,
                                              double sum) {
  constexpr int kLanes = kFp8Block / VE;  // of a block
  constexpr uint32_t kNear = 2;           // fp32 steps
  uint8_t* q = static_cast<uint8_t*>(a.y) + r * a.ldy;
  const Rstd rs(sum, a);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float w[VE], y[VE];
    weight.get(col, j, w);
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      y[e] = rs.times(v[j][e], w[e]);
      if (col.counts(j, e)) top = abs_bits(y[e]) > top ? abs_bits(y[e]) : top;
    }
    top = max_of_16<kLanes == 32>(top);
    if constexpr (POW2) {
      const bool near = top < kInfBits && (top & 0x7fffffu) - (0x600000u - kNear) <= 2 * kNear;
      if (__any(near)) {
        double big = 0.0;
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (col.counts(j, e)) big = fmax(big, fabs(double(v[j][e]) * rs.exact * w[e]));
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) big = fmax(big, __shfl_xor(big, off, 64));
        // times 448 it stays on its side of the power of two
        if (near) top = abs_bits(float(big / kFp8Max) * kFp8Max);
      }
    }
    if (!col.live(j)) continue;
    const BlockScale<POW2> s(top);
    store_fp8<POW2, VE>(q + col.at[j], s, y, col.skip[j], a.h - col.at[j]);
    if (lane % kLanes == 0) s.store(a.scales, int64_t((lane + j * stride) / kLanes) * a.lds + r);
  }
}

template <class T, int WPR, int EPL, bool FULL, bool STREAM, bool FP8>
__global__ void __launch_bounds__(norm_threads(WPR, kFwdThreads), FP8 && EPL <= 24 ? 4 : 1)
    rmsnorm_fwd_kernel(RmsFwd a) {
  // x, residual, sum and y may share rows: a row is in registers before any of it is written
  constexpr bool kHold = WPR < 16 && (FP8 || !STREAM);
  constexpr int VE = Elem<T>::kVec, NV = EPL / VE, RG = norm_threads(WPR, kFwdThreads) / (64 * WPR);
  __shared__ double red[2][norm_threads(WPR, kFwdThreads) / 64];
  const int lane = threadIdx.x % (64 * WPR), group = threadIdx.x / (64 * WPR);
  const float fh = float(a.h);
  const T* x = static_cast<const T*>(a.x);
  const T* add = static_cast<const T*>(a.residual);
  const Columns<VE, NV, 64 * WPR, FULL> col(lane, a.h);
  const Weight<T, Columns<VE, NV, 64 * WPR, FULL>, VE, NV, kHold> weight(col, a.weight, a.wide);
  const int64_t step = int64_t(gridDim.x) * RG;
  int64_t r = int64_t(blockIdx.x) * RG + group;
  raw4 next[NV], nadd[NV];  // the row after the one being worked on
  auto fetch = [&](int64_t row) {
    row = row < a.n ? row : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) next[j] = col.template load<STREAM>(x + row * a.ldx, j);
    if (add) {
#pragma unroll
      for (int j = 0; j < NV; ++j) nadd[j] = col.template load<STREAM>(add + row * a.ldr, j);
    }
  };
  fetch(r);
  int parity = 0;
  for (int64_t base = int64_t(blockIdx.x) * RG; base < a.n; base += step, r += step) {
    float v[NV][VE];
#pragma unroll
    for (int j = 0; j < NV; ++j) Elem<T>::unpack(next[j], v[j]);
    if (add) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float b[VE];
        Elem<T>::unpack(nadd[j], b);
#pragma unroll
        for (int q = 0; q < VE; ++q) v[j][q] += b[q];
        Elem<T>::unpack(Elem<T>::pack(v[j]), v[j]);  // what is kept is what is normalised
      }
    }
    if (base + step < a.n) fetch(r + step);
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < VE; ++q) s += col.counts(j, q) ? v[j][q] * v[j][q] : 0.f;
    const double sum = row_sum_f64<WPR>(s, red[parity]);
    parity ^= 1;
    const float rstd = 1.f / sqrtf(float(sum) / fh + a.eps);
    if (r >= a.n) continue;
    if (a.sum) {
      T* sr = static_cast<T*>(a.sum) + r * a.ldsum;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (col.live(j)) col.template store<STREAM>(sr, j, v[j]);
    }
    if constexpr (FP8) {
      if (a.pow2)
        store_row_fp8<true, T>(col, a, r, lane, 64 * WPR, v, weight, sum);
      else
        store_row_fp8<false, T>(col, a, r, lane, 64 * WPR, v, weight, sum);
    } else {
      T* yr = static_cast<T*>(a.y) + r * a.ldy;
      const Rstd rs(sum, a);  // fp32 rows: the numbers that the 8-bit form rounds
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float w[VE];
        weight.get(col, j, w);
#pragma unroll
        for (int q = 0; q < VE; ++q)
          w[q] = sizeof(T) == 4 ? rs.times_any(v[j][q], w[q]) : v[j][q] * rstd * w[q];
        if (col.live(j)) col.template store<STREAM>(yr, j, w);
      }
    }
    if (lane == 0 && a.rstd) a.rstd[r] = rstd;
  }
}

struct RmsBwd {
  const void *grad, *x, *weight, *grad_sum;
  const float* rstd;
  int64_t n, ldg, ldx, ldgs, lddx;
  int h;
  bool wide;
  void* dx;
  float* part;  // partial rows of dw, or NULL
};

// With the workgroup's partial row of dw, where a.part is given.
template <class T, int WPR, int EPL, bool FULL>
__global__ void __launch_bounds__(norm_threads(WPR, kBwdThreads)) rmsnorm_bwd_kernel(RmsBwd a) {
  // grad, grad_sum and dx may be the same rows
  constexpr int VE = Elem<T>::kVec, NV = EPL / VE, RG = norm_threads(WPR, kBwdThreads) / (64 * WPR);
  __shared__ float red[2][norm_threads(WPR, kBwdThreads) / 64][1];
  const int lane = threadIdx.x % (64 * WPR), group = threadIdx.x / (64 * WPR);
  const float inv_h = 1.f / float(a.h);
  const T* g = static_cast<const T*>(a.grad);
  const T* x = static_cast<const T*>(a.x);
  const T* gs = static_cast<const T*>(a.grad_sum);
  T* dx = static_cast<T*>(a.dx);
  const Columns<VE, NV, 64 * WPR, FULL> col(lane, a.h);
  const Weight<T, Columns<VE, NV, 64 * WPR, FULL>, VE, NV, true> weight(col, a.weight, a.wide);
  float dw[NV][VE] = {};
  const int64_t step = int64_t(gridDim.x) * RG;
  int64_t r = int64_t(blockIdx.x) * RG + group;
  raw4 nx[NV], ng[NV], ns[NV];  // the row after the one being worked on
  float nrs;
  auto fetch = [&](int64_t row) {
    row = row < a.n ? row : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) nx[j] = col.load(x + row * a.ldx, j);
#pragma unroll
    for (int j = 0; j < NV; ++j) ng[j] = col.load(g + row * a.ldg, j);
    if (gs) {
#pragma unroll
      for (int j = 0; j < NV; ++j) ns[j] = col.load(gs + row * a.ldgs, j);
    }
    nrs = a.rstd[row];
  };
  fetch(r);
  int parity = 0;
  for (int64_t base = int64_t(blockIdx.x) * RG; base < a.n; base += step, r += step) {
    const bool live = r < a.n;
    const float rs = nrs;
    float xh[NV][VE], u[NV][VE];
    raw4 keep[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Elem<T>::unpack(nx[j], xh[j]);
      Elem<T>::unpack(ng[j], u[j]);
      keep[j] = ns[j];
    }
    if (base + step < a.n) fetch(r + step);
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[VE];
      weight.get(col, j, w);
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        xh[j][q] *= rs;
        if (live) dw[j][q] += u[j][q] * xh[j][q];
        u[j][q] *= w[q];
        s[0] += col.counts(j, q) ? u[j][q] * xh[j][q] : 0.f;
      }
    }
    row_sums<WPR, 1>(s, red[parity]);
    parity ^= 1;
    if (!live || !dx) continue;
    const float b = s[0] * inv_h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!col.live(j)) continue;
#pragma unroll
      for (int q = 0; q < VE; ++q) u[j][q] = rs * (u[j][q] - xh[j][q] * b);
      if (gs) {
        float k[VE];
        Elem<T>::unpack(keep[j], k);
#pragma unroll
        for (int q = 0; q < VE; ++q) u[j][q] += k[q];
      }
      col.store(dx + r * a.lddx, j, u[j]);
    }
  }
  if (!a.part) return;
  // this workgroup's partial row: its row groups added through LDS, in group order
  if constexpr (RG > 1) {
    constexpr int LANES = 64 * WPR;
    __shared__ float sums[RG - 1][EPL][LANES];
    if (group > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < VE; ++q) sums[group - 1][j * VE + q][lane] = dw[j][q];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int k = 0; k < RG - 1; ++k)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < VE; ++q) dw[j][q] += sums[k][j * VE + q][lane];
  }
  float* pw = a.part + int64_t(blockIdx.x) * a.h;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (col.skip[j] == 0 && (FULL || a.h >= VE)) {
      store_some<float, VE>(pw + col.at[j], VE, dw[j]);
    } else if (!FULL && col.live(j)) {  // the row's last vector, or a row shorter than one
#pragma unroll
      for (int q = 0; q < VE; ++q)
        if (col.counts(j, q)) pw[col.at[j] + q] = dw[j][q];
    }
  }
}

// Rows past kRegRowOf: no sums of dw, and the row is widened anew for each of its two uses, since 32
// numbers a lane of x and grad with the next row's do not fit the registers of sixteen wavefronts
// ([4096, 20000] bf16 with the gradient of the sum: 146 us beside the 90 of its columns, and 287 as
// the shorter rows are done).
template <class T, int WPR, int EPL, bool FULL>
__global__ void __launch_bounds__(64 * WPR) rmsnorm_bwd_long_kernel(RmsBwd a) {
  constexpr int VE = Elem<T>::kVec, NV = EPL / VE;
  __shared__ float red[2][WPR][1];
  const int lane = threadIdx.x;
  const float inv_h = 1.f / float(a.h);
  const T* gs = static_cast<const T*>(a.grad_sum);
  const Columns<VE, NV, 64 * WPR, FULL> col(lane, a.h);
  int parity = 0;
  for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
    raw4 x[NV], g[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j] = col.load(static_cast<const T*>(a.x) + r * a.ldx, j);
#pragma unroll
    for (int j = 0; j < NV; ++j) g[j] = col.load(static_cast<const T*>(a.grad) + r * a.ldg, j);
    const float rs = a.rstd[r];
    // x · rstd and grad · weight of vector j
    auto widen = [&](int j, float(&xh)[VE], float(&u)[VE]) {
      float w[VE];
      weight_at<T>(col, a.weight, a.wide, j, w);
      asm volatile("" : "+v"(x[j]), "+v"(g[j]));
      Elem<T>::unpack(x[j], xh);
      Elem<T>::unpack(g[j], u);
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        xh[q] *= rs;
        u[q] *= w[q];
      }
    };
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float xh[VE], u[VE];
      widen(j, xh, u);
#pragma unroll
      for (int q = 0; q < VE; ++q) s[0] += col.counts(j, q) ? u[q] * xh[q] : 0.f;
    }
    row_sums<WPR, 1>(s, red[parity]);
    parity ^= 1;
    const float b = s[0] * inv_h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!col.live(j)) continue;
      float xh[VE], u[VE], k[VE] = {};
      if (gs) Elem<T>::unpack(col.load(gs + r * a.ldgs, j), k);
      widen(j, xh, u);
#pragma unroll
      for (int q = 0; q < VE; ++q) u[q] = rs * (u[q] - xh[q] * b) + k[q];
      T* to = static_cast<T*>(a.dx) + r * a.lddx;
      if (FULL || col.skip[j] == 0) {
        col.store(to, j, u);
      } else {  // the row's last vector: what grad_sum holds there may still be read by its owner
#pragma unroll
        for (int q = 0; q < VE; ++q)
          if (col.counts(j, q)) to[col.at[j] + q] = Elem<T>::from_f32(u[q]);
      }
    }
  }
}

// dw of long rows: a workgroup adds the rows blockIdx.y, blockIdx.y + gridDim.y, ... of its 256
// vectors of columns into partial row blockIdx.y.
constexpr int kColBatch = 4;  // rows in flight per lane
template <class T>
__global__ void __launch_bounds__(256) rms_columns_kernel(const T* __restrict__ g, int64_t ldg,
                                                          const T* __restrict__ x, int64_t ldx,
                                                          const float* __restrict__ rstd,
                                                          int64_t n, int64_t h,
                                                          float* __restrict__ part) {
  constexpr int VE = Elem<T>::kVec;
  const int64_t col = (int64_t(blockIdx.x) * 256 + threadIdx.x) * VE;
  if (col >= h) return;
  const int64_t cnt = h - col;
  float dw[VE] = {};
  for (int64_t r0 = blockIdx.y; r0 < n; r0 += int64_t(kColBatch) * gridDim.y) {
    float xs[kColBatch][VE], gr[kColBatch][VE], rs[kColBatch];
#pragma unroll
    for (int k = 0; k < kColBatch; ++k) {
      const int64_t r = r0 + int64_t(k) * gridDim.y;
      if (r >= n) continue;
      load_some<T, VE>(x + r * ldx + col, cnt, xs[k]);
      load_some<T, VE>(g + r * ldg + col, cnt, gr[k]);
      rs[k] = rstd[r];
    }
#pragma unroll
    for (int k = 0; k < kColBatch; ++k) {
      if (r0 + int64_t(k) * gridDim.y >= n) break;
#pragma unroll
      for (int q = 0; q < VE; ++q) dw[q] += gr[k][q] * (xs[k][q] * rs[k]);
    }
  }
  float* pw = part + int64_t(blockIdx.y) * h + col;
#pragma unroll
  for (int q = 0; q < VE; ++q)
    if (q < cnt) pw[q] = dw[q];
}

template <class T, bool FP8>
hipError_t run_fwd(const RmsFwd& a, hipStream_t s) {
  return with_shape<kFwdElems>(a.h, [&](auto wpr, auto epl) {
    constexpr int WPR = decltype(wpr)::value, EPL = decltype(epl)::value;
    constexpr int RG = norm_threads(WPR, kFwdThreads) / (64 * WPR);
    const int64_t grid = std::min<int64_t>((a.n + RG - 1) / RG,
                                           kFwdGrid * 512 / norm_threads(WPR, kFwdThreads));
    const int64_t moved = a.n * a.h * int64_t(sizeof(T)) * (a.residual ? 4 : 2);
    TimedLaunch t(s, FP8 ? K_RMS_FP8_FWD : K_RMS_FWD);
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(norm_threads(WPR, kFwdThreads)), 0, s,
                         a);
    };
    if (a.h % Elem<T>::kVec != 0)
      launch(rmsnorm_fwd_kernel<T, WPR, EPL, false, false, FP8>);
    else if (moved <= kStreamBytes)
      launch(rmsnorm_fwd_kernel<T, WPR, EPL, true, false, FP8>);
    else
      launch(rmsnorm_fwd_kernel<T, WPR, EPL, true, true, FP8>);
    return hipGetLastError();
  });
}

template <class T>
hipError_t run_bwd_rows(const RmsBwd& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  if (a.h > kRegRowOf<T>) {
    if (a.part) {
      constexpr int VE = Elem<T>::kVec;
      TimedLaunch t(s, K_RMS_BWD);
      hipLaunchKernelGGL((rms_columns_kernel<T>),
                         dim3(unsigned((a.h + 256 * VE - 1) / (256 * VE)),
                              unsigned(part_rows<T>(a.n, a.h))),
                         dim3(256), 0, s, static_cast<const T*>(a.grad), a.ldg,
                         static_cast<const T*>(a.x), a.ldx, a.rstd, a.n, int64_t(a.h), a.part);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (!a.dx) return hipSuccess;  // the long rows' kernel writes it without a test
  }
  return with_shape<kBwdElems>(a.h, [&](auto wpr, auto epl) {
    constexpr int WPR = decltype(wpr)::value, EPL = decltype(epl)::value;
    constexpr int RG = norm_threads(WPR, kBwdThreads) / (64 * WPR);
    constexpr bool PARAMS = 64 * WPR * EPL <= kRegRowOf<T>;
    const int64_t grid = std::min<int64_t>((a.n + RG - 1) / RG, PARAMS ? bwd_grid(a.h) : kLongGrid);
    TimedLaunch t(s, K_RMS_BWD);
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(norm_threads(WPR, kBwdThreads)), 0, s,
                         a);
    };
    if constexpr (!PARAMS) {
      if (a.h % Elem<T>::kVec == 0)
        launch(rmsnorm_bwd_long_kernel<T, WPR, EPL, true>);
      else
        launch(rmsnorm_bwd_long_kernel<T, WPR, EPL, false>);
    } else {
      if (a.h % Elem<T>::kVec == 0)
        launch(rmsnorm_bwd_kernel<T, WPR, EPL, true>);
      else
        launch(rmsnorm_bwd_kernel<T, WPR, EPL, false>);
    }
    return hipGetLastError();
  });
}

// Partial rows that run_bwd_rows() leaves.
template <class T>
int64_t rows_left(int64_t n, int64_t h) {
  if (n == 0 || h > kRegRowOf<T>) return part_rows<T>(n, h);
  int64_t rows = 0;
  (void)with_shape<kBwdElems>(h, [&](auto wpr, auto) {
    constexpr int WPR = decltype(wpr)::value;
    constexpr int RG = norm_threads(WPR, kBwdThreads) / (64 * WPR);
    rows = std::min<int64_t>((n + RG - 1) / RG, bwd_grid(h));
    return hipSuccess;
  });
  return rows;
}

}  // namespace

hipError_t rmsnorm_fwd_run(const RmsFwdArgs& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  const RmsFwd k{a.x,   a.residual, a.weight,       a.n,      a.ldx,      a.ldr,
                 int(a.h), a.param_dtype == kF32, a.eps, a.y, a.residual_out, a.ldy,
                 a.ldro, a.rstd_out, a.scales,      a.lds,    a.scale_dtype == kScaleE8M0};
  const bool fp8 = a.scales != nullptr;
  switch (a.dtype) {
    case kBF16: return fp8 ? run_fwd<Bf16, true>(k, s) : run_fwd<Bf16, false>(k, s);
    case kF16: return fp8 ? run_fwd<_Float16, true>(k, s) : run_fwd<_Float16, false>(k, s);
    default: return fp8 ? run_fwd<float, true>(k, s) : run_fwd<float, false>(k, s);
  }
}

size_t rmsnorm_workspace_bytes(int64_t n, int64_t h) {
  // the 16-bit types' partial rows are no fewer than fp32's
  return std::max<size_t>(align256(size_t(part_rows<Bf16>(n, h)) * size_t(h) * 4), 256);
}

hipError_t rmsnorm_bwd_run(const RmsBwdArgs& a, hipStream_t s) {
  const bool add = a.flags & RMSNORM_ACCUMULATE;
  if (!a.grad_x && !a.grad_weight) return hipSuccess;  // neither gradient is asked for
  if (a.n == 0 && (!a.grad_weight || add)) return hipSuccess;
  float* part = a.grad_weight ? static_cast<float*>(a.workspace) : nullptr;
  const RmsBwd k{a.grad, a.x,    a.weight, a.grad_residual, a.rstd, a.n,
                 a.ldg,  a.ldx,  a.ldgr,   a.lddx,          int(a.h), a.param_dtype == kF32,
                 a.grad_x, part};
  hipError_t e;
  switch (a.dtype) {
    case kBF16: e = run_bwd_rows<Bf16>(k, s); break;
    case kF16: e = run_bwd_rows<_Float16>(k, s); break;
    default: e = run_bwd_rows<float>(k, s);
  }
  if (e != hipSuccess || !part) return e;
  const int64_t rows = a.dtype == kF32 ? rows_left<float>(a.n, a.h) : rows_left<Bf16>(a.n, a.h);
  switch (a.grad_param_dtype) {
    case kBF16: return run_reduce<Bf16>(part, nullptr, rows, a.h, add, a.grad_weight, nullptr, s);
    case kF16:
      return run_reduce<_Float16>(part, nullptr, rows, a.h, add, a.grad_weight, nullptr, s);
    default: return run_reduce<float>(part, nullptr, rows, a.h, add, a.grad_weight, nullptr, s);
  }
}

}  // namespace lce
