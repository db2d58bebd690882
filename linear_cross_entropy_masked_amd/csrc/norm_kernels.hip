// Layer norm forward and backward for gfx950.
//
//   forward   y = (x − μ) · r · w + b,  μ = mean(x),  r = 1 / sqrt(mean((x − μ)²) + eps)  per row
//   backward  u = g · w,  x̂ = (x − μ) · r
//             dx = r · (u − mean(u) − x̂ · mean(u · x̂))            per row
//             dw (=|+=) Σ_rows g · x̂,   db (=|+=) Σ_rows g
//
// Memory-bound: 2 · n · h elements move in the forward ([32768, 8192] bf16: 187 us in short runs, 5.8
// TB/s, where a copy of 2 GiB reaches 4.9; in an unbroken run of forty the launches take 188 to 230),
// 3 · n · h in the backward ([8192, 4096] bf16: 48 us, 4.2 TB/s, 44 of them in the rows' kernel; what
// is left is the partial rows below and the start of each workgroup). A row lives in
// the registers of WPR wavefronts (at most 32 elements a lane) from its one read to its one
// write; the mean is known before the squares are summed, so the variance does not cancel. Rows
// are dealt to a fixed grid, each lane loading the next row's vectors before the sums of this. In
// the backward every lane keeps the columns it owns for all of its rows and adds their dw and db
// terms in fp32 registers (the longest rows take a pass of their own for them, norm_columns_kernel);
// each workgroup writes one partial row of each, and param_reduce_kernel adds those in workgroup
// order (no atomics: a result does not change from run to run).
#include <algorithm>

#include "common.h"
#include "elem.h"
#include "norm_rows.h"
#include "ops.h"

namespace lce {

namespace {

// Launch shapes, measured on the [32768, 8192] bf16 forward and the [8192, 4096] bf16 and
// [4099, 2051] fp16 backward: the forward takes rows in workgroups of at least 512 threads with
// 32 elements a lane (190 us; 256 threads 206, 16 elements 200), the backward in workgroups of
// at least 256 threads with 16 or 24 (50 and 27 us; 512 threads and 32 elements 55 and 50: its
// running dw and db take two registers an element, and fewer rows are in flight at once).
constexpr int kFwdThreads = 512, kFwdElems = 32;
constexpr int kBwdThreads = 256, kBwdElems = 16;
constexpr int64_t kFwdGrid = 2048;
// Workgroups of the backward, each of which costs one partial row of dw and of db: two per CU of
// 256 threads (768 or 1024 of them: [8192, 4096] 47 or 55 against 47 us, [4099, 2051] fp16 28 or 30
// against 23), one of 512 ([4096, 8192] 52 us, two 58), four where the partial rows are short
// ([60000, 257] 34 us, two 42; [16384, 512] 19 either way). Past kRegRow elements a row's dw and db
// do not fit the registers of a workgroup beside the row: they are summed by columns, in kColRows
// groups of rows ([1024, 20011] bf16 110 us so and 254 in the rows' own pass).
constexpr int64_t kShortRow = 512, kPairRow = 256 * 24, kRegRow = 512 * 32;
constexpr int64_t kColRows = 64;
int64_t bwd_grid(int64_t h) { return h <= kShortRow ? 1024 : h <= kPairRow ? 512 : 256; }
int64_t part_rows(int64_t n, int64_t h) {
  return std::min(n, h > kRegRow ? kColRows : bwd_grid(h));
}
// A forward of whole vectors that moves more than this passes by the caches (non-temporal loads
// and stores): 1 GiB takes 188 us so and 199 without, 256 MiB 54 either way, 128 MiB 31 so and
// 28 without.
constexpr int64_t kStreamBytes = int64_t(512) << 20;

template <class T, class P, int WPR, int EPL, bool FULL, bool STREAM>
__global__ void __launch_bounds__(norm_threads(WPR, kFwdThreads)) layernorm_fwd_kernel(
    const T* x, int64_t n, int h, int64_t ldx, const P* __restrict__ weight,
    const P* __restrict__ bias, float eps, T* y, int64_t ldy, float* __restrict__ mean_out,
    float* __restrict__ rstd_out) {
  // x and y may be the same rows: a row is in registers before any of it is written
  constexpr int VE = Elem<T>::kVec, NV = EPL / VE, RG = norm_threads(WPR, kFwdThreads) / (64 * WPR);
  __shared__ float red[2][norm_threads(WPR, kFwdThreads) / 64][1];
  const int lane = threadIdx.x % (64 * WPR), group = threadIdx.x / (64 * WPR);
  const float fh = float(h);
  const Columns<VE, NV, 64 * WPR, FULL> col(lane, h);
  const int64_t step = int64_t(gridDim.x) * RG;
  int64_t r = int64_t(blockIdx.x) * RG + group;
  raw4 next[NV];  // the row after the one being worked on
#pragma unroll
  for (int j = 0; j < NV; ++j) next[j] = col.template load<STREAM>(x + (r < n ? r : 0) * ldx, j);
  for (int64_t base = int64_t(blockIdx.x) * RG; base < n; base += step, r += step) {
    float v[NV][VE];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) Elem<T>::unpack(next[j], v[j]);
    if (base + step < n) {
      const T* xn = x + (r + step < n ? r + step : 0) * ldx;
#pragma unroll
      for (int j = 0; j < NV; ++j) next[j] = col.template load<STREAM>(xn, j);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < VE; ++q) s[0] += col.counts(j, q) ? v[j][q] : 0.f;
    row_sums<WPR, 1>(s, red[0]);
    const float mean = s[0] / fh;  // divided, not multiplied by 1 / h: exact for a constant row
    float ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        v[j][q] -= mean;
        ss[0] += col.counts(j, q) ? v[j][q] * v[j][q] : 0.f;
      }
    row_sums<WPR, 1>(ss, red[1]);
    const float rstd = 1.f / sqrtf(ss[0] / fh + eps);
    if (r >= n) continue;
    T* yr = y + r * ldy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!col.live(j)) continue;
      float w[VE], b[VE];
      col.param(weight, j, 1.f, w);
      col.param(bias, j, 0.f, b);
#pragma unroll
      for (int q = 0; q < VE; ++q) w[q] = v[j][q] * rstd * w[q] + b[q];
      col.template store<STREAM>(yr, j, w);
    }
    if (lane == 0) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
  }
}

// PARAMS: with the workgroup's partial rows of dw and db, where part_w is given.
template <class T, class P, int WPR, int EPL, bool FULL, bool PARAMS>
__global__ void __launch_bounds__(norm_threads(WPR, kBwdThreads)) layernorm_bwd_kernel(
    const T* g, int64_t ldg, const T* __restrict__ x, int64_t ldx, const float* __restrict__ mean,
    const float* __restrict__ rstd, const P* __restrict__ weight, int64_t n, int h, T* dx,
    int64_t lddx, float* __restrict__ part_w, float* __restrict__ part_b) {
  // g and dx may be the same rows, as x and y in the forward
  constexpr int VE = Elem<T>::kVec, NV = EPL / VE, RG = norm_threads(WPR, kBwdThreads) / (64 * WPR);
  __shared__ float red[2][norm_threads(WPR, kBwdThreads) / 64][2];
  const int lane = threadIdx.x % (64 * WPR), group = threadIdx.x / (64 * WPR);
  const float inv_h = 1.f / float(h);
  const Columns<VE, NV, 64 * WPR, FULL> col(lane, h);
  float dw[NV][VE] = {}, db[NV][VE] = {};
  const int64_t step = int64_t(gridDim.x) * RG;
  int64_t r = int64_t(blockIdx.x) * RG + group;
  raw4 nx[NV], ng[NV];  // the row after the one being worked on
  float nmu, nrs;
  auto fetch = [&](int64_t row) {
    row = row < n ? row : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) nx[j] = col.load(x + row * ldx, j);
#pragma unroll
    for (int j = 0; j < NV; ++j) ng[j] = col.load(g + row * ldg, j);
    nmu = mean[row];
    nrs = rstd[row];
  };
  fetch(r);
  int parity = 0;
  for (int64_t base = int64_t(blockIdx.x) * RG; base < n; base += step, r += step) {
    const bool live = r < n;
    const float mu = nmu, rs = nrs;
    float xh[NV][VE], u[NV][VE];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Elem<T>::unpack(nx[j], xh[j]);
      Elem<T>::unpack(ng[j], u[j]);
    }
    if (base + step < n) fetch(r + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float w[VE];
      col.param(weight, j, 1.f, w);
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        xh[j][q] = (xh[j][q] - mu) * rs;
        if (PARAMS && live) {
          dw[j][q] += u[j][q] * xh[j][q];
          db[j][q] += u[j][q];
        }
        u[j][q] *= w[q];
        s[0] += col.counts(j, q) ? u[j][q] : 0.f;
        s[1] += col.counts(j, q) ? u[j][q] * xh[j][q] : 0.f;
      }
    }
    row_sums<WPR, 2>(s, red[parity]);
    parity ^= 1;
    if (!live || !dx) continue;
    const float a = s[0] * inv_h, b = s[1] * inv_h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!col.live(j)) continue;
#pragma unroll
      for (int q = 0; q < VE; ++q) u[j][q] = rs * (u[j][q] - a - xh[j][q] * b);
      col.store(dx + r * lddx, j, u[j]);
    }
  }
  if (!PARAMS || !part_w) return;
  // this workgroup's partial rows: its row groups added through LDS, in group order
  if constexpr (RG > 1) {
    constexpr int LANES = 64 * WPR;
    __shared__ float sums[RG - 1][2 * EPL][LANES];
    if (group > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          sums[group - 1][j * VE + q][lane] = dw[j][q];
          sums[group - 1][EPL + j * VE + q][lane] = db[j][q];
        }
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int k = 0; k < RG - 1; ++k)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int q = 0; q < VE; ++q) {
          dw[j][q] += sums[k][j * VE + q][lane];
          db[j][q] += sums[k][EPL + j * VE + q][lane];
        }
  }
  float* pw = part_w + int64_t(blockIdx.x) * h;
  float* pb = part_b + int64_t(blockIdx.x) * h;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (col.skip[j] == 0 && (FULL || h >= VE)) {
      store_some<float, VE>(pw + col.at[j], VE, dw[j]);
      store_some<float, VE>(pb + col.at[j], VE, db[j]);
    } else if (!FULL && col.live(j)) {  // the row's last vector, or a row shorter than one
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        if (!col.counts(j, q)) continue;
        pw[col.at[j] + q] = dw[j][q];
        pb[col.at[j] + q] = db[j][q];
      }
    }
  }
}

// dw and db of long rows: a workgroup adds the rows blockIdx.y, blockIdx.y + gridDim.y, ... of its
// 256 vectors of columns into partial row blockIdx.y.
constexpr int kColBatch = 4;  // rows in flight per lane
template <class T>
__global__ void __launch_bounds__(256) norm_columns_kernel(
    const T* __restrict__ g, int64_t ldg, const T* __restrict__ x, int64_t ldx,
    const float* __restrict__ mean, const float* __restrict__ rstd, int64_t n, int64_t h,
    float* __restrict__ part_w, float* __restrict__ part_b) {
  constexpr int VE = Elem<T>::kVec;
  const int64_t col = (int64_t(blockIdx.x) * 256 + threadIdx.x) * VE;
  if (col >= h) return;
  const int64_t cnt = h - col;
  float dw[VE] = {}, db[VE] = {};
  for (int64_t r0 = blockIdx.y; r0 < n; r0 += int64_t(kColBatch) * gridDim.y) {
    float xs[kColBatch][VE], gs[kColBatch][VE], mu[kColBatch], rs[kColBatch];
#pragma unroll
    for (int k = 0; k < kColBatch; ++k) {
      const int64_t r = r0 + int64_t(k) * gridDim.y;
      if (r >= n) continue;
      load_some<T, VE>(x + r * ldx + col, cnt, xs[k]);
      load_some<T, VE>(g + r * ldg + col, cnt, gs[k]);
      mu[k] = mean[r];
      rs[k] = rstd[r];
    }
#pragma unroll
    for (int k = 0; k < kColBatch; ++k) {
      if (r0 + int64_t(k) * gridDim.y >= n) break;
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        dw[q] += gs[k][q] * ((xs[k][q] - mu[k]) * rs[k]);
        db[q] += gs[k][q];
      }
    }
  }
  float* pw = part_w + int64_t(blockIdx.y) * h + col;
  float* pb = part_b + int64_t(blockIdx.y) * h + col;
#pragma unroll
  for (int q = 0; q < VE; ++q) {
    if (q >= cnt) break;
    pw[q] = dw[q];
    pb[q] = db[q];
  }
}

template <class T, class P>
hipError_t run_fwd(const NormFwdArgs& a, hipStream_t s) {
  return with_shape<kFwdElems>(a.h, [&](auto wpr, auto epl) {
    constexpr int WPR = decltype(wpr)::value, EPL = decltype(epl)::value;
    constexpr int RG = norm_threads(WPR, kFwdThreads) / (64 * WPR);
    const int64_t grid = std::min<int64_t>((a.n + RG - 1) / RG, kFwdGrid);
    TimedLaunch t(s, K_NORM_FWD);
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(norm_threads(WPR, kFwdThreads)), 0, s,
                         static_cast<const T*>(a.x), a.n, int(a.h), a.ldx,
                         static_cast<const P*>(a.weight), static_cast<const P*>(a.bias), a.eps,
                         static_cast<T*>(a.y), a.ldy, a.mean_out, a.rstd_out);
    };
    if (a.h % Elem<T>::kVec != 0)
      launch(layernorm_fwd_kernel<T, P, WPR, EPL, false, false>);
    else if (2 * a.n * a.h * int64_t(sizeof(T)) <= kStreamBytes)
      launch(layernorm_fwd_kernel<T, P, WPR, EPL, true, false>);
    else
      launch(layernorm_fwd_kernel<T, P, WPR, EPL, true, true>);
    return hipGetLastError();
  });
}

template <class T, class P>
hipError_t run_bwd_rows(const NormBwdArgs& a, float* part_w, float* part_b, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  if (a.h > kRegRow && part_w) {
    constexpr int VE = Elem<T>::kVec;
    TimedLaunch t(s, K_NORM_BWD);
    hipLaunchKernelGGL((norm_columns_kernel<T>),
                       dim3(unsigned((a.h + 256 * VE - 1) / (256 * VE)),
                            unsigned(part_rows(a.n, a.h))),
                       dim3(256), 0, s, static_cast<const T*>(a.grad), a.ldg,
                       static_cast<const T*>(a.x), a.ldx, a.mean, a.rstd, a.n, a.h, part_w,
                       part_b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.grad_x) return e;
  }
  return with_shape<kBwdElems>(a.h, [&](auto wpr, auto epl) {
    constexpr int WPR = decltype(wpr)::value, EPL = decltype(epl)::value;
    constexpr int RG = norm_threads(WPR, kBwdThreads) / (64 * WPR);
    constexpr bool PARAMS = 64 * WPR * EPL <= kRegRow;
    const int64_t grid = std::min<int64_t>((a.n + RG - 1) / RG, bwd_grid(a.h));
    TimedLaunch t(s, K_NORM_BWD);
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(norm_threads(WPR, kBwdThreads)), 0, s,
                         static_cast<const T*>(a.grad), a.ldg, static_cast<const T*>(a.x), a.ldx,
                         a.mean, a.rstd, static_cast<const P*>(a.weight), a.n, int(a.h),
                         static_cast<T*>(a.grad_x), a.lddx, part_w, part_b);
    };
    if (a.h % Elem<T>::kVec == 0)
      launch(layernorm_bwd_kernel<T, P, WPR, EPL, true, PARAMS>);
    else
      launch(layernorm_bwd_kernel<T, P, WPR, EPL, false, PARAMS>);
    return hipGetLastError();
  });
}

// Partial rows that run_bwd_rows() leaves.
int64_t rows_left(int64_t n, int64_t h) {
  if (n == 0 || h > kRegRow) return part_rows(n, h);
  int64_t rows = 0;
  with_shape<kBwdElems>(h, [&](auto wpr, auto) {
    constexpr int WPR = decltype(wpr)::value;
    constexpr int RG = norm_threads(WPR, kBwdThreads) / (64 * WPR);
    rows = std::min<int64_t>((n + RG - 1) / RG, bwd_grid(h));
    return hipSuccess;
  });
  return rows;
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
  const int64_t rows = part_rows(n, h);
  return std::max<size_t>(2 * align256(size_t(rows) * size_t(h) * 4), 256);
}

hipError_t layernorm_bwd_run(const NormBwdArgs& a, hipStream_t s) {
  const bool params = a.grad_weight || a.grad_bias;
  if (a.n == 0 && (!params || (a.flags & LAYERNORM_ACCUMULATE))) return hipSuccess;
  float *pw = nullptr, *pb = nullptr;
  if (params) {
    pw = static_cast<float*>(a.workspace);
    pb = reinterpret_cast<float*>(static_cast<char*>(a.workspace) +
                                  align256(size_t(part_rows(a.n, a.h)) * size_t(a.h) * 4));
  }
  const int64_t rows = rows_left(a.n, a.h);
  const bool wide = a.param_dtype == kF32;
  hipError_t e;
  switch (a.dtype) {
    case kBF16:
      e = wide ? run_bwd_rows<Bf16, float>(a, pw, pb, s)
               : run_bwd_rows<Bf16, Bf16>(a, pw, pb, s);
      break;
    case kF16:
      e = wide ? run_bwd_rows<_Float16, float>(a, pw, pb, s)
               : run_bwd_rows<_Float16, _Float16>(a, pw, pb, s);
      break;
    default: e = run_bwd_rows<float, float>(a, pw, pb, s);
  }
  if (e != hipSuccess || !params) return e;
  const bool add = a.flags & LAYERNORM_ACCUMULATE;
  switch (a.grad_param_dtype) {
    case kBF16: return run_reduce<Bf16>(pw, pb, rows, a.h, add, a.grad_weight, a.grad_bias, s);
    case kF16: return run_reduce<_Float16>(pw, pb, rows, a.h, add, a.grad_weight, a.grad_bias, s);
    default: return run_reduce<float>(pw, pb, rows, a.h, add, a.grad_weight, a.grad_bias, s);
  }
}

}  // namespace lce
