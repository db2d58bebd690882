// Layer norm forward and backward for gfx950.
//
//   forward   y = (x − μ) · r · w + b,  μ = mean(x),  r = 1 / sqrt(mean((x − μ)²) + eps)  per row
//   backward  u = g · w,  x̂ = (x − μ) · r
//             dx = r · (u − mean(u) − x̂ · mean(u · x̂))            per row
//             dw (=|+=) Σ_rows g · x̂,   db (=|+=) Σ_rows g
//
// Memory-bound: 2 · n · h elements move in the forward, 3 · n · h in the backward. A row lives in
// the registers of WPR wavefronts (at most 32 elements a lane) from its one read to its one
// write; the mean is known before the squares are summed, so the variance does not cancel. Rows
// are dealt to a fixed grid. In the backward every lane keeps the columns it owns for all of its
// rows and adds their dw and db terms in fp32 registers; each workgroup writes one partial row
// of each, and param_reduce_kernel adds those in workgroup order (no atomics: a result does not
// change from run to run).
#include <algorithm>

#include "common.h"
#include "elem.h"
#include "ops.h"

namespace lce {

namespace {

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}

// Threads of a workgroup for rows of WPR wavefronts.
constexpr int norm_threads(int wpr) { return wpr > 8 ? 64 * wpr : 512; }

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

template <class T, class P, int WPR, int EPL>
__global__ void __launch_bounds__(norm_threads(WPR)) layernorm_fwd_kernel(
    const T* x, int64_t n, int64_t h, int64_t ldx, const P* __restrict__ weight,
    const P* __restrict__ bias, float eps, T* y, int64_t ldy, float* __restrict__ mean_out,
    float* __restrict__ rstd_out) {
  // x and y may be the same rows: a row is in registers before any of it is written
  constexpr int VE = Elem<T>::kVec, NV = EPL / VE, RG = norm_threads(WPR) / (64 * WPR);
  __shared__ float red[2][norm_threads(WPR) / 64][1];
  const int lane = threadIdx.x % (64 * WPR), group = threadIdx.x / (64 * WPR);
  const float fh = float(h);
  for (int64_t base = int64_t(blockIdx.x) * RG; base < n; base += int64_t(gridDim.x) * RG) {
    const int64_t r = base + group;
    const bool live = r < n;
    const T* xr = x + (live ? r : 0) * ldx;
    float v[NV][VE];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = int64_t(lane + j * 64 * WPR) * VE;
      if (c < h) {
        load_some<T, VE>(xr + c, h - c, v[j]);
      } else {
#pragma unroll
        for (int q = 0; q < VE; ++q) v[j][q] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < VE; ++q) s[0] += v[j][q];
    row_sums<WPR, 1>(s, red[0]);
    const float mean = s[0] / fh;  // divided, not multiplied by 1 / h: exact for a constant row
    float ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = int64_t(lane + j * 64 * WPR) * VE;
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        v[j][q] -= mean;
        if (c + q < h) ss[0] += v[j][q] * v[j][q];
      }
    }
    row_sums<WPR, 1>(ss, red[1]);
    const float rstd = 1.f / sqrtf(ss[0] / fh + eps);
    if (!live) continue;
    T* yr = y + r * ldy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = int64_t(lane + j * 64 * WPR) * VE;
      if (c >= h) continue;
      float w[VE], b[VE];
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        w[q] = 1.f;
        b[q] = 0.f;
      }
      if (weight) load_some<P, VE>(weight + c, h - c, w);
      if (bias) load_some<P, VE>(bias + c, h - c, b);
#pragma unroll
      for (int q = 0; q < VE; ++q) w[q] = v[j][q] * rstd * w[q] + b[q];
      store_some<T, VE>(yr + c, h - c, w);
    }
    if (lane == 0) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
  }
}

template <class T, class P, int WPR, int EPL>
__global__ void __launch_bounds__(norm_threads(WPR)) layernorm_bwd_kernel(
    const T* g, int64_t ldg, const T* __restrict__ x, int64_t ldx, const float* __restrict__ mean,
    const float* __restrict__ rstd, const P* __restrict__ weight, int64_t n, int64_t h, T* dx,
    int64_t lddx, float* __restrict__ part_w, float* __restrict__ part_b) {
  // g and dx may be the same rows, as x and y in the forward
  constexpr int VE = Elem<T>::kVec, NV = EPL / VE, RG = norm_threads(WPR) / (64 * WPR);
  __shared__ float red[2][norm_threads(WPR) / 64][2];
  const int lane = threadIdx.x % (64 * WPR), group = threadIdx.x / (64 * WPR);
  const float inv_h = 1.f / float(h);
  float dw[NV][VE] = {}, db[NV][VE] = {};
  int parity = 0;
  for (int64_t base = int64_t(blockIdx.x) * RG; base < n; base += int64_t(gridDim.x) * RG) {
    const int64_t r = base + group;
    const bool live = r < n;
    const float mu = live ? mean[r] : 0.f, rs = live ? rstd[r] : 0.f;
    float xh[NV][VE], u[NV][VE];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = int64_t(lane + j * 64 * WPR) * VE;
#pragma unroll
      for (int q = 0; q < VE; ++q) xh[j][q] = u[j][q] = 0.f;
      if (live && c < h) {
        load_some<T, VE>(x + r * ldx + c, h - c, xh[j]);
        load_some<T, VE>(g + r * ldg + c, h - c, u[j]);
      }
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = int64_t(lane + j * 64 * WPR) * VE;
      float w[VE];
#pragma unroll
      for (int q = 0; q < VE; ++q) w[q] = 1.f;
      if (weight && c < h) load_some<P, VE>(weight + c, h - c, w);
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        xh[j][q] = (xh[j][q] - mu) * rs;
        dw[j][q] += u[j][q] * xh[j][q];
        db[j][q] += u[j][q];
        u[j][q] *= w[q];
        s[0] += u[j][q];
        s[1] += u[j][q] * xh[j][q];
      }
    }
    row_sums<WPR, 2>(s, red[parity]);
    parity ^= 1;
    if (!live || !dx) continue;
    const float a = s[0] * inv_h, b = s[1] * inv_h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = int64_t(lane + j * 64 * WPR) * VE;
      if (c >= h) continue;
#pragma unroll
      for (int q = 0; q < VE; ++q) u[j][q] = rs * (u[j][q] - a - xh[j][q] * b);
      store_some<T, VE>(dx + r * lddx + c, h - c, u[j]);
    }
  }
  if (!part_w) return;
  // this workgroup's partial rows: its row groups one after the other
  float* pw = part_w + int64_t(blockIdx.x) * h;
  float* pb = part_b + int64_t(blockIdx.x) * h;
  for (int k = 0; k < RG; ++k) {
    if (RG > 1) __syncthreads();
    if (group != k) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = int64_t(lane + j * 64 * WPR) * VE;
      if (c >= h) continue;
      float t[VE];
      if (k > 0) {
#pragma unroll
        for (int q = 0; q < VE; ++q) t[q] = c + q < h ? pw[c + q] : 0.f;
#pragma unroll
        for (int q = 0; q < VE; ++q) dw[j][q] += t[q];
#pragma unroll
        for (int q = 0; q < VE; ++q) t[q] = c + q < h ? pb[c + q] : 0.f;
#pragma unroll
        for (int q = 0; q < VE; ++q) db[j][q] += t[q];
      }
      store_some<float, VE>(pw + c, h - c, dw[j]);
      store_some<float, VE>(pb + c, h - c, db[j]);
    }
  }
}

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

constexpr int64_t kFwdGrid = 2048;  // workgroups the forward's rows are dealt to
constexpr int64_t kBwdGrid = 256;   // workgroups of the backward: one partial row each

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Calls f with the row shape (WPR, EPL) for rows of h elements: 32 elements a lane, fewer where
// one wavefront holds the row with fewer; wavefronts per row doubled until the row fits.
template <class F>
hipError_t with_shape(int64_t h, F&& f) {
  using std::integral_constant;
  if (h <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 8>{});
  if (h <= 1024) return f(integral_constant<int, 1>{}, integral_constant<int, 16>{});
  if (h <= 2048) return f(integral_constant<int, 1>{}, integral_constant<int, 32>{});
  if (h <= 4096) return f(integral_constant<int, 2>{}, integral_constant<int, 32>{});
  if (h <= 8192) return f(integral_constant<int, 4>{}, integral_constant<int, 32>{});
  if (h <= 16384) return f(integral_constant<int, 8>{}, integral_constant<int, 32>{});
  return f(integral_constant<int, 16>{}, integral_constant<int, 32>{});
}

template <class T, class P>
hipError_t run_fwd(const NormFwdArgs& a, hipStream_t s) {
  return with_shape(a.h, [&](auto wpr, auto epl) {
    constexpr int WPR = decltype(wpr)::value, EPL = decltype(epl)::value;
    constexpr int RG = norm_threads(WPR) / (64 * WPR);
    const int64_t grid = std::min<int64_t>((a.n + RG - 1) / RG, kFwdGrid);
    TimedLaunch t(s, K_NORM_FWD);
    hipLaunchKernelGGL((layernorm_fwd_kernel<T, P, WPR, EPL>), dim3(unsigned(grid)),
                       dim3(norm_threads(WPR)), 0, s, static_cast<const T*>(a.x), a.n, a.h, a.ldx,
                       static_cast<const P*>(a.weight), static_cast<const P*>(a.bias), a.eps,
                       static_cast<T*>(a.y), a.ldy, a.mean_out, a.rstd_out);
    return hipGetLastError();
  });
}

template <class T, class P>
hipError_t run_bwd_rows(const NormBwdArgs& a, float* part_w, float* part_b, int64_t* rows,
                        hipStream_t s) {
  return with_shape(a.h, [&](auto wpr, auto epl) {
    constexpr int WPR = decltype(wpr)::value, EPL = decltype(epl)::value;
    constexpr int RG = norm_threads(WPR) / (64 * WPR);
    const int64_t grid = std::min<int64_t>((a.n + RG - 1) / RG, kBwdGrid);
    *rows = grid;
    if (grid == 0) return hipSuccess;
    TimedLaunch t(s, K_NORM_BWD);
    hipLaunchKernelGGL((layernorm_bwd_kernel<T, P, WPR, EPL>), dim3(unsigned(grid)),
                       dim3(norm_threads(WPR)), 0, s, static_cast<const T*>(a.grad), a.ldg,
                       static_cast<const T*>(a.x), a.ldx, a.mean, a.rstd,
                       static_cast<const P*>(a.weight), a.n, a.h, static_cast<T*>(a.grad_x),
                       a.lddx, part_w, part_b);
    return hipGetLastError();
  });
}

template <class P>
hipError_t run_reduce(const NormBwdArgs& a, const float* pw, const float* pb, int64_t rows,
                      hipStream_t s) {
  const dim3 grid(unsigned((a.h + kRedCols - 1) / kRedCols), 2);
  TimedLaunch t(s, K_NORM_PARAM_REDUCE);
  if (a.flags & LAYERNORM_ACCUMULATE)
    hipLaunchKernelGGL((param_reduce_kernel<P, true>), grid, dim3(kRedCols * kRedGroups), 0, s, pw,
                       pb, rows, a.h, static_cast<P*>(a.grad_weight),
                       static_cast<P*>(a.grad_bias));
  else
    hipLaunchKernelGGL((param_reduce_kernel<P, false>), grid, dim3(kRedCols * kRedGroups), 0, s,
                       pw, pb, rows, a.h, static_cast<P*>(a.grad_weight),
                       static_cast<P*>(a.grad_bias));
  return hipGetLastError();
}

}  // namespace

hipError_t layernorm_fwd_run(const NormFwdArgs& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  const bool wide = a.param_dtype == kF32;
  switch (a.dtype) {
    case kBF16: return wide ? run_fwd<Bf16, float>(a, s) : run_fwd<Bf16, Bf16>(a, s);
    case kF16: return wide ? run_fwd<_Float16, float>(a, s) : run_fwd<_Float16, _Float16>(a, s);
    default: return run_fwd<float, float>(a, s);
  }
}

size_t layernorm_workspace_bytes(int64_t n, int64_t h) {
  const int64_t rows = std::min(n, kBwdGrid);
  return std::max<size_t>(2 * align256(size_t(rows) * size_t(h) * 4), 256);
}

hipError_t layernorm_bwd_run(const NormBwdArgs& a, hipStream_t s) {
  const bool params = a.grad_weight || a.grad_bias;
  if (a.n == 0 && (!params || (a.flags & LAYERNORM_ACCUMULATE))) return hipSuccess;
  float *pw = nullptr, *pb = nullptr;
  if (params) {
    pw = static_cast<float*>(a.workspace);
    pb = reinterpret_cast<float*>(static_cast<char*>(a.workspace) +
                                  align256(size_t(std::min(a.n, kBwdGrid)) * size_t(a.h) * 4));
  }
  int64_t rows = 0;
  const bool wide = a.param_dtype == kF32;
  hipError_t e;
  switch (a.dtype) {
    case kBF16:
      e = wide ? run_bwd_rows<Bf16, float>(a, pw, pb, &rows, s)
               : run_bwd_rows<Bf16, Bf16>(a, pw, pb, &rows, s);
      break;
    case kF16:
      e = wide ? run_bwd_rows<_Float16, float>(a, pw, pb, &rows, s)
               : run_bwd_rows<_Float16, _Float16>(a, pw, pb, &rows, s);
      break;
    default: e = run_bwd_rows<float, float>(a, pw, pb, &rows, s);
  }
  if (e != hipSuccess || !params) return e;
  switch (a.grad_param_dtype) {
    case kBF16: return run_reduce<Bf16>(a, pw, pb, rows, s);
    case kF16: return run_reduce<_Float16>(a, pw, pb, rows, s);
    default: return run_reduce<float>(a, pw, pb, rows, s);
  }
}

}  // namespace lce
