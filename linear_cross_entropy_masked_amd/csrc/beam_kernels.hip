// One step of a beam search for gfx950: the best continuations of each batch entry's beams, and
// its states put in the order of their beams.
//
//   candidate (j, v): score_j + (z_jv − lse_j),  lse_j = log Σ_v exp(z_jv)
//
// taken best first, equal scores in the order (beam, logit, token). Two launches:
//   rows  a workgroup holds a slice of one row of logits in registers, so that the row is read
//         once for its maximum, its sum of exponentials and its best logits. The threads' own
//         maxima give a threshold that at least `num` of them reach, which few logits do: those
//         are put in LDS and ranked by counting. Where too many do (ties in plenty), the slice's
//         best are taken one at a time.
//   pick  a workgroup per batch entry: a wavefront merges a row's slices in the same way, then
//         every candidate counts the better ones of each row by bisection.
// The rows' launch is bound by reading the logits: 32 x 8 rows of 128256 in bf16 17.8 us, 3.7 TB/s
// (torch's sums of as many rows take 23 us, its maxima 38; kernels here that only read reach 5.1 to
// 6.7 TB/s over longer times); the numbers held as stored, so that eight wavefronts share a SIMD, and
// one operation a term made that of 25.9. The pick takes 8.2 us there
// (16 slices of 16 candidates a row) and 5.5 for 4 rows of 32777: a chain of loads, a threshold by
// bits and a bisection.
// Sums of exponentials are fp32 within a slice's threads, fp64 across slices, and scores are
// compared in fp64. No atomics decide an order: the lists are filled by atomics and ranked by
// keys that are all different.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "elem.h"
#include "ops.h"

namespace lce {

namespace {

constexpr int kThreads = 256;
constexpr int kHolders = 96;  // threads of a slice whose logits are looked through
constexpr int kList = 256;    // candidates of a slice that are ranked at once
constexpr int kRowList = 440; // the same of a row
constexpr int kMost = BEAM_MAX_CANDIDATES;
constexpr int kPairs = 880;   // candidates of an entry whose ranks fit one wavefront's list
static_assert(kPairs * 4 <= kRowList * 8, "ranks take a list's place");

// Floats as integers of the same order; 0 is below all of them.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
// A logit above minus infinity and its token as one key, better ones larger; 0: none.
__device__ __forceinline__ uint64_t key_of(float z, uint32_t token) {
  return uint64_t(ordered(z)) << 32 | uint32_t(~token);
}

// join() over the wavefront's values, the result in all lanes; no step goes through LDS.
template <class F>
__device__ __forceinline__ uint32_t wave_join(uint32_t x, F&& join) {
  auto lanes = [&](auto ctrl) {
    constexpr int CTRL = decltype(ctrl)::value;
    x = join(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CTRL, 0xf, 0xf, true)));
  };
  lanes(std::integral_constant<int, 0xB1>{});   // lane ^ 1
  lanes(std::integral_constant<int, 0x4E>{});   // lane ^ 2
  lanes(std::integral_constant<int, 0x141>{});  // mirrored within 8
  lanes(std::integral_constant<int, 0x140>{});  // mirrored within 16
  const auto r = __builtin_amdgcn_permlane16_swap(int(x), int(x), false, false);
  x = join(uint32_t(r[0]), uint32_t(r[1]));
  const auto h = __builtin_amdgcn_permlane32_swap(int(x), int(x), false, false);
  return join(uint32_t(h[0]), uint32_t(h[1]));
}
__device__ __forceinline__ float wave_max(float x) {
  return __uint_as_float(wave_join(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_add(float x) {
  return __uint_as_float(wave_join(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// A threshold that at least `want` of the wavefront's PER · 64 values reach (0 where there are
// not so many), and not many more than that where the values differ. Bits are fixed from the first
// in which any two values differ, until the number that reaches it is at most want + want / 4.
template <int PER>
__device__ __forceinline__ uint32_t threshold(const uint32_t (&x)[PER], int want) {
  if (want > 64 * PER) return 0;
  uint32_t lo = x[0], hi = x[0];
#pragma unroll
  for (int k = 1; k < PER; ++k) {
    lo = x[k] < lo ? x[k] : lo;
    hi = x[k] > hi ? x[k] : hi;
  }
  hi = __builtin_amdgcn_readfirstlane(
      wave_join(hi, [](uint32_t a, uint32_t b) { return a > b ? a : b; }));
  lo = __builtin_amdgcn_readfirstlane(
      wave_join(lo, [](uint32_t a, uint32_t b) { return a < b ? a : b; }));
  int bit = 31 - __clz(int(hi ^ lo));  // -1: all the same
  uint32_t t = bit < 0 ? hi : hi >> 1 >> bit << bit << 1;
  for (; bit >= 0; --bit) {
    const uint32_t c = t | 1u << bit;
    int reach = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) reach += __popcll(__ballot(x[k] >= c));
    if (reach >= want) {
      t = c;
      if (reach <= want + want / 4) break;
    }
  }
  return t;
}

struct RowsK {
  const void* logits;
  int64_t v, ld;
  uint32_t splits;
  int num;
  uint64_t* keys;   // [rows, splits, num], best first, 0 where there are fewer
  float2* sums;     // [rows, splits]: maximum, sum of exp(z − maximum)
};

// Eight logits of a thread as they are stored; minus infinity behind the row's end.
template <class T>
struct Logits8 {
  static constexpr int kRaws = 8 / Elem<T>::kVec;
  raw4 r[kRaws];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int k = 0; k < kRaws; ++k) r[k] = load_raw(p + k * Elem<T>::kVec);
  }
  __device__ __forceinline__ void load_some(const T* p, int64_t cnt) {
    if (cnt >= 8) return load(p);
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = q < cnt ? Elem<T>::to_f32(p[q]) : -INFINITY;
#pragma unroll
    for (int k = 0; k < kRaws; ++k) {
      float y[Elem<T>::kVec];
#pragma unroll
      for (int q = 0; q < Elem<T>::kVec; ++q) y[q] = x[k * Elem<T>::kVec + q];
      r[k] = Elem<T>::pack(y);
    }
  }
  // Widened anew each time: kept, the numbers would take twice the registers.
  __device__ __forceinline__ void get(float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < kRaws; ++k) {
      asm volatile("" : "+v"(r[k]));
      float y[Elem<T>::kVec];
      Elem<T>::unpack(r[k], y);
#pragma unroll
      for (int q = 0; q < Elem<T>::kVec; ++q) x[k * Elem<T>::kVec + q] = y[q];
    }
  }
};

template <class T, int EPT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 8 : 5) beam_rows_kernel(RowsK a) {
  constexpr int NV = EPT / 8, kWaves = kThreads / 64;
  __shared__ float top[kThreads];
  __shared__ float wave_m[kWaves], wave_s[kWaves];
  __shared__ uint32_t limit;
  __shared__ int holders, count;
  // the logits of the threads whose largest reaches the threshold, and where each one's start
  __shared__ __attribute__((aligned(16))) float held[kHolders][EPT];
  __shared__ int from_thread[kHolders];
  __shared__ uint64_t list[kList];
  __shared__ uint64_t best[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t row = blockIdx.x / a.splits, split = blockIdx.x - row * a.splits;
  const int64_t base = int64_t(split) * (kThreads * EPT), at = base + tid * 8;
  const T* z = static_cast<const T*>(a.logits) + int64_t(row) * a.ld;
  // as they are stored, widened where they are used: half the registers for 16-bit types, which
  // lets eight wavefronts share a SIMD instead of five
  using Vec = Logits8<T>;
  Vec raw[NV];
  if (base + kThreads * EPT <= a.v) {
#pragma unroll
    for (int j = 0; j < NV; ++j) raw[j].load(z + at + j * kThreads * 8);
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = at + int64_t(j) * kThreads * 8;
      raw[j].load_some(z + c, a.v - c);
    }
  }
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float x[8];
    raw[j].get(x);
#pragma unroll
    for (int q = 0; q < 8; ++q) m = fmaxf(m, x[q]);
  }
  m += 0.f;  // one zero: -0 becomes +0
  const float mine = m;
  top[tid] = m;
  if (tid == 0) holders = count = 0;
  // The sum of exp(x - m) about the thread's own maximum m, each as 2^(x · L - c) with L = log2 e
  // and c = m · L rounded: one operation instead of two. What the rounding of c makes of all terms
  // alike is taken out of their sum, r = m · L - c being exact; 2^r is near 1 up to |m| = 2^20
  // (|r| up to 2^-4), and further out the difference x - m comes first.
  float s = 0.f;
  const bool any = m > -INFINITY;
  if (__any(any && fabsf(m) > 0x1p20f)) {
    const float from = any ? m : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[8];
      raw[j].get(x);
#pragma unroll
      for (int q = 0; q < 8; ++q) s += fast_exp2((x[q] - from) * kLog2e);
    }
  } else {
    const float from = any ? m : 0.f, c = from * kLog2e;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[8];
      raw[j].get(x);
#pragma unroll
      for (int q = 0; q < 8; ++q) s += fast_exp2(fmaf(x[q], kLog2e, -c));
    }
    s *= fast_exp2(-fmaf(from, kLog2e, -c));
  }
  const bool bad = __any(!(s >= 0.f));  // a NaN or +inf: the sum says so, whatever it meets
  const float wm = wave_max(m);
  s = wave_add(any ? s * fast_exp2((m - wm) * kLog2e) : 0.f);
  if (lane == 0) {
    wave_m[wave] = wm;
    wave_s[wave] = bad ? NAN : s;
  }
  __syncthreads();
  if (wave == 0) {
    uint32_t t[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) t[w] = ordered(top[64 * w + lane]);
    const uint32_t lim = threshold<kWaves>(t, a.num);
    // no logit at or below minus infinity is a candidate
    if (lane == 0) limit = lim > ordered(-INFINITY) ? lim : ordered(-INFINITY) + 1;
  } else if (wave == 1 && lane == 0) {
    float gm = wave_m[0], gs = wave_s[0];
    bool nan = !(gs >= 0.f);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      nan |= !(wave_s[w] >= 0.f);
      lse_merge(gm, gs, wave_m[w], wave_s[w]);
    }
    a.sums[blockIdx.x] = float2{gm, nan ? NAN : gs};
  }
  __syncthreads();
  const float lim = from_ordered(limit);
  if (mine >= lim) {
    const int p = atomicAdd(&holders, 1);
    if (p < kHolders) {
      from_thread[p] = tid;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[8];
        raw[j].get(x);
#pragma unroll
        for (int q = 0; q < 8; ++q) held[p][j * 8 + q] = x[q];
      }
    }
  }
  __syncthreads();
  const int h = holders;
  uint64_t* out = a.keys + int64_t(blockIdx.x) * a.num;
  if (h <= kHolders) {
    for (int i = tid; i < h * EPT; i += kThreads) {
      const float v = held[i / EPT][i % EPT];
      if (v >= lim) {
        const int p = atomicAdd(&count, 1);
        const int e = i % EPT;
        if (p < kList)
          list[p] = key_of(v + 0.f, uint32_t(base + (e / 8 * kThreads + from_thread[i / EPT]) * 8 +
                                             e % 8));
      }
    }
    __syncthreads();
    const int c = count;
    if (c <= kList) {
      if (tid < c) {
        const uint64_t k = list[tid];
        int rank = 0;
        for (int i = 0; i < c; ++i) rank += list[i] > k;
        if (rank < a.num) out[rank] = k;
      }
      if (tid >= c && tid < a.num) out[tid] = 0;
      return;
    }
  }
  // one at a time: the best key below the last one taken
  uint64_t last = ~uint64_t(0);
  for (int r = 0; r < a.num; ++r) {
    uint64_t k = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[8];
      raw[j].get(x);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (x[q] > -INFINITY) {
          const uint64_t e = key_of(x[q] + 0.f, uint32_t(at + j * kThreads * 8 + q));
          if (e < last && e > k) k = e;
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const uint64_t o = __shfl_xor((unsigned long long)k, off, 64);
      k = o > k ? o : k;
    }
    if (lane == 0) best[wave] = k;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) k = best[w] > k ? best[w] : k;
    if (tid == 0) out[r] = k;
    last = k;
    __syncthreads();
    // nothing is left: what follows is 0 too, since no key is below 0
  }
}

struct PickK {
  const float* scores;
  const uint8_t* finished;
  const uint64_t* keys;
  const float2* sums;
  int64_t splits;
  int beams, num;
  int32_t eos, ignore_index;
  float* scores_out;
  int32_t *parents_out, *tokens_out;
  uint8_t* finished_out;
  int32_t* status_out;
};

// What the wavefront's lanes wrote to LDS is there for all of them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// The best `num` keys of n at `in`, in order, into the wavefront's `out` (LDS); 0 behind the last.
// `have`: the lane's first kHeld keys, at in[place(lane, 0)], in[place(lane, 1)], ...
// A row's keys are its slices' lists, each in order: a lane that took every 64th of them would hold
// the same few ranks of all lists, one lane all of the best, and the threshold that enough lanes
// reach would let most keys pass (4 x 16 rows of 46491 x 32 candidates: 216 us, one key at a time).
// So each 64 are turned by kTurn lanes against the 64 before.
constexpr int kHeld = 8, kTurn = 21;
__device__ __forceinline__ int64_t place(int lane, int64_t k) {
  return 64 * k + ((lane + kTurn * uint32_t(k)) & 63);
}
__device__ __forceinline__ void merge_row(const uint64_t* in, int64_t n,
                                          const uint64_t (&have)[kHeld], int num, uint64_t* list,
                                          int* count, uint64_t* out) {
  const int lane = threadIdx.x & 63;
  uint32_t top[1] = {0};
  auto each = [&](auto&& f) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) f(have[k]);
    for (int64_t k0 = kHeld; 64 * k0 < n; k0 += kHeld) {
      uint64_t x[kHeld];
#pragma unroll
      for (int k = 0; k < kHeld; ++k) x[k] = place(lane, k0 + k) < n ? in[place(lane, k0 + k)] : 0;
#pragma unroll
      for (int k = 0; k < kHeld; ++k) f(x[k]);
    }
  };
  each([&](uint64_t k) { top[0] = uint32_t(k >> 32) > top[0] ? uint32_t(k >> 32) : top[0]; });
  const uint32_t lim = threshold<1>(top, num);
  if (lane == 0) *count = 0;
  wave_sync();
  each([&](uint64_t k) {
    if (k != 0 && uint32_t(k >> 32) >= lim) {
      const int p = atomicAdd(count, 1);
      if (p < kRowList) list[p] = k;
    }
  });
  wave_sync();
  const int c = *static_cast<volatile int*>(count);
  for (int r = lane; r < num; r += 64)
    if (r >= c) out[r] = 0;
  if (c <= kRowList) {
    for (int i = lane; i < c; i += 64) {
      const uint64_t k = list[i];
      int rank = 0;
      for (int o = 0; o < c; ++o) rank += list[o] > k;
      if (rank < num) out[rank] = k;
    }
  } else {
    uint64_t last = ~uint64_t(0);
    for (int r = 0; r < num; ++r) {
      uint64_t k = 0;
      each([&](uint64_t e) {
        if (e < last && e > k) k = e;
      });
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)k, off, 64);
        k = o > k ? o : k;
      }
      if (lane == 0) out[r] = k;
      last = k;
    }
  }
  wave_sync();
}

// Workgroup b: batch entry b. LDS: scores, tokens and ranks [beams, num], a list per wavefront.
__global__ void __launch_bounds__(512) beam_pick_kernel(PickK a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int all = a.beams * a.num;
  double* score = reinterpret_cast<double*>(lds);
  uint64_t* lists = reinterpret_cast<uint64_t*>(score + all);
  uint64_t* sorted = lists + waves * kRowList;
  int32_t* token = reinterpret_cast<int32_t*>(sorted + waves * kMost);
  int* counts = token + all;
  int* found = counts + waves;               // candidates there are
  int* ranks = reinterpret_cast<int*>(lists);  // up to kPairs, once the lists are merged
  const int64_t b = blockIdx.x;
  if (threadIdx.x == 0) *found = 0;
  for (int j = wave; j < a.beams; j += waves) {
    const int64_t row = b * a.beams + j, n = a.splits * a.num;
    const float acc = a.scores[row];
    const bool done = a.finished && a.finished[row];
    double* sj = score + j * a.num;
    int32_t* tj = token + j * a.num;
    const float2* ms = a.sums + row * a.splits;
    const uint64_t* in = a.keys + row * n;
    // everything that comes from memory is asked for at once
    const float2 own = lane < a.splits ? ms[lane] : float2{-INFINITY, 0.f};
    uint64_t have[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) have[k] = place(lane, k) < n ? in[place(lane, k)] : 0;
    // the row's logsumexp, lanes in order of their distance
    float m = own.x;
    bool nan = !(own.y >= 0.f) || own.x == INFINITY;
    for (int64_t i = lane + 64; i < a.splits; i += 64) m = fmaxf(m, ms[i].x);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    double s = own.x > -INFINITY ? double(own.y) * exp(double(own.x) - double(m)) : 0.0;
    for (int64_t i = lane + 64; i < a.splits; i += 64) {
      const float2 p = ms[i];
      nan |= !(p.y >= 0.f) || p.x == INFINITY;
      if (p.x > -INFINITY) s += double(p.y) * exp(double(p.x) - double(m));
    }
    s = wave_sum_f64(s);
    const bool bad = __any(nan) || !(acc < INFINITY);  // a NaN or +inf among the logits or scores
    if ((done ? !(acc < INFINITY) : bad) && a.status_out && lane == 0)
      atomicOr(a.status_out, LCE_STATUS_BAD_LOGITS);
    if (done) {
      for (int r = lane; r < a.num; r += 64) {
        sj[r] = r == 0 && acc < INFINITY ? double(acc) : -INFINITY;
        tj[r] = a.eos;
      }
      continue;
    }
    if (bad || !(m > -INFINITY) || !(acc > -INFINITY)) {
      for (int r = lane; r < a.num; r += 64) sj[r] = -INFINITY;
      continue;
    }
    uint64_t* out = sorted + wave * kMost;
    merge_row(in, n, have, a.num, lists + wave * kRowList, counts + wave, out);
    const double log_s = log(s);  // not added to m, beside which it may be lost
    for (int r = lane; r < a.num; r += 64) {
      const uint64_t k = out[r];
      const double z = from_ordered(uint32_t(k >> 32));
      sj[r] = k ? double(acc) + (z - double(m) - log_s) : -INFINITY;
      tj[r] = int32_t(~uint32_t(k));
    }
  }
  __syncthreads();
  // how many of beam i come before candidate p of another: better ones, and equal ones of an
  // earlier beam. A beam's are in order, so they are found by bisection.
  auto before = [&](int p, int i) {
    const double s = score[p];
    int lo = 0, hi = a.num;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      const double o = score[i * a.num + mid];
      if (o > s || (o == s && i < p / a.num))
        lo = mid + 1;
      else
        hi = mid;
    }
    return lo;
  };
  const int64_t to = b * a.num;
  auto put = [&](int p, int rank) {
    if (rank >= a.num) return;
    const int j = p / a.num;
    const int32_t tok = token[p];
    a.scores_out[to + rank] = float(score[p]);
    a.parents_out[to + rank] = j;
    a.tokens_out[to + rank] = tok;
    if (a.finished_out)
      a.finished_out[to + rank] =
          (a.finished && a.finished[b * a.beams + j]) || (a.eos >= 0 && tok == a.eos);
  };
  if (all <= kPairs) {  // a thread takes a candidate and another beam at a time
    for (int p = threadIdx.x; p < all; p += blockDim.x) {
      ranks[p] = p % a.num;  // those of its own beam
      if (score[p] > -INFINITY) atomicAdd(found, 1);
    }
    __syncthreads();
    for (int u = threadIdx.x; u < all * a.beams; u += blockDim.x) {
      const int p = u % all, i = u / all;
      if (i == p / a.num || !(score[p] > -INFINITY)) continue;
      const int n = before(p, i);
      if (n > 0) atomicAdd(ranks + p, n);
    }
    __syncthreads();
    for (int p = threadIdx.x; p < all; p += blockDim.x)
      if (score[p] > -INFINITY) put(p, ranks[p]);
  } else {  // too many for their ranks to be held
    for (int p = threadIdx.x; p < all; p += blockDim.x) {
      if (!(score[p] > -INFINITY)) continue;
      atomicAdd(found, 1);
      int rank = p % a.num;
      for (int i = 0; i < a.beams && rank < a.num; ++i)
        if (i != p / a.num) rank += before(p, i);
      put(p, rank);
    }
    __syncthreads();
  }
  for (int r = threadIdx.x; r < a.num; r += blockDim.x) {
    if (r < *found) continue;
    a.scores_out[to + r] = -INFINITY;
    a.parents_out[to + r] = -1;
    a.tokens_out[to + r] = a.ignore_index;
    if (a.finished_out) a.finished_out[to + r] = 0;
  }
}

// ------------------------------------------------------------------------------- states

// Copies: 3.5 GB read and written in 641 us, 5.4 TB/s (a large copy: 4.9).
constexpr int kStates = 16;         // of a launch
constexpr int kChunk = 16384;       // bytes of a segment that a workgroup copies
constexpr int kTile = 32768;        // bytes of LDS where states are reordered in place

struct StatesK {
  lce_beam_state st[kStates];
  int64_t first[kStates + 1];  // the first workgroup of each
  int64_t chunks[kStates];     // of a segment
  int count;
  const int32_t* parents;
  int64_t beams, slots;
  int64_t chunk;
};

typedef uint32_t raw4_b1 __attribute__((ext_vector_type(4), aligned(1)));

__device__ __forceinline__ void copy_bytes(char* to, const char* from, int64_t bytes) {
  for (int64_t o = int64_t(threadIdx.x) * 16; o < bytes; o += kThreads * 16) {
    if (o + 16 <= bytes) {
      const raw4 v = from ? raw4(*reinterpret_cast<const raw4_b1*>(from + o)) : raw4{0, 0, 0, 0};
      *reinterpret_cast<raw4_b1*>(to + o) = v;
    } else {
      for (int64_t i = o; i < bytes; ++i) to[i] = from ? from[i] : 0;
    }
  }
}

// Workgroup: a chunk of one segment of one slot, copied from its parent's.
__global__ void __launch_bounds__(kThreads) beam_copy_kernel(StatesK a) {
  int t = 0;
  while (int64_t(blockIdx.x) >= a.first[t + 1]) ++t;
  const lce_beam_state& st = a.st[t];
  int64_t u = int64_t(blockIdx.x) - a.first[t];
  const int64_t chunk = u % a.chunks[t];
  u /= a.chunks[t];
  const int64_t seg = u % st.segments;
  u /= st.segments;
  const int64_t slot = u % a.slots, b = u / a.slots;
  const int32_t p = a.parents[b * a.slots + slot];
  const int64_t at = chunk * a.chunk;
  const int64_t left = st.segment_bytes - at, bytes = left < a.chunk ? left : a.chunk;
  const char* from = nullptr;
  if (p >= 0 && p < a.beams)
    from = static_cast<const char*>(st.in) + b * st.in_entry + p * st.in_beam +
           seg * st.in_segment + at;
  copy_bytes(static_cast<char*>(st.out) + b * st.out_entry + slot * st.out_beam +
                 seg * st.out_segment + at,
             from, bytes);
}

// In place: a workgroup takes the same bytes of all of an entry's beams through LDS, reads those
// that another slot wants and writes those that change. Beams are copied one after another, so few
// bytes are in flight where many share the LDS: eight states [16, k, 1000, 1024] in bf16 take 114, 308
// and 956 us at 2, 4 and 8 beams (176, 328 and 638 into other tensors), [8, 16, 1000, 1024] 2.1 ms
// (0.64) and [2, 64, 1000, 1024] 21 ms (0.65).
__global__ void __launch_bounds__(kThreads) beam_inplace_kernel(StatesK a) {
  __shared__ __attribute__((aligned(16))) char tile[kTile];
  int t = 0;
  while (int64_t(blockIdx.x) >= a.first[t + 1]) ++t;
  const lce_beam_state& st = a.st[t];
  int64_t u = int64_t(blockIdx.x) - a.first[t];
  const int64_t chunk = u % a.chunks[t];
  u /= a.chunks[t];
  const int64_t seg = u % st.segments, b = u / st.segments;
  const int32_t* parents = a.parents + b * a.beams;
  const int64_t at = chunk * a.chunk;
  const int64_t left = st.segment_bytes - at, bytes = left < a.chunk ? left : a.chunk;
  char* base = static_cast<char*>(st.out) + b * st.out_entry + seg * st.out_segment + at;
  for (int j = 0; j < a.beams; ++j) {
    bool wanted = false;
    for (int i = 0; i < a.beams; ++i) wanted |= i != j && parents[i] == j;
    if (wanted) copy_bytes(tile + j * a.chunk, base + j * st.out_beam, bytes);
  }
  __syncthreads();
  for (int j = 0; j < a.beams; ++j) {
    const int32_t p = parents[j];
    if (p == j) continue;
    copy_bytes(base + j * st.out_beam, p >= 0 && p < a.beams ? tile + p * a.chunk : nullptr, bytes);
  }
}

// Logits of a slice. Long ones leave the pick less (32 x 8 rows of 128256 x 16 candidates: rows and
// pick 17.8 + 9.2 us in slices of 8192, 23.1 + 17.9 of 4096, 32.8 + 36.9 of 2048), short ones
// spread few rows over the CUs: the longest of which there are 512. Asking for 1024, 512 and 256 of
// them takes 44, 32 and 31 us for 4 x 16 rows of 46491 x 32 candidates, 29.7, 23.2 and 22.7 for
// 2 x 16 of 118257 x 16, 15.4, 16.4 and 16.5 for 16 x 8 of 32777 x 8.
int64_t slice_of(int64_t rows, int64_t v) {
  if (rows * ((v + 8191) / 8192) >= 512) return 8192;
  if (rows * ((v + 4095) / 4096) >= 512) return 4096;
  return 2048;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

template <class T>
hipError_t run_rows(const RowsK& k, int64_t rows, int64_t slice, hipStream_t s) {
  TimedLaunch t(s, K_BEAM_ROWS);
  const dim3 grid(unsigned(rows * k.splits));
  if (slice == 8192)
    hipLaunchKernelGGL((beam_rows_kernel<T, 32>), grid, dim3(kThreads), 0, s, k);
  else if (slice == 4096)
    hipLaunchKernelGGL((beam_rows_kernel<T, 16>), grid, dim3(kThreads), 0, s, k);
  else
    hipLaunchKernelGGL((beam_rows_kernel<T, 8>), grid, dim3(kThreads), 0, s, k);
  return hipGetLastError();
}

}  // namespace

int64_t beam_step_slices(int64_t rows, int64_t v) {
  const int64_t slice = slice_of(rows, v);
  return rows * ((v + slice - 1) / slice);
}

size_t beam_step_workspace_bytes(int64_t batch, int64_t beams, int64_t v, int64_t num) {
  const size_t slices = size_t(beam_step_slices(batch * beams, v));
  return align256(slices * size_t(num) * 8) + align256(slices * 8);
}

hipError_t beam_step_run(const BeamStepArgs& a, hipStream_t s) {
  if (a.batch == 0) return hipSuccess;
  const int64_t rows = a.batch * a.beams, slice = slice_of(rows, a.v);
  const int64_t splits = (a.v + slice - 1) / slice;
  uint64_t* keys = static_cast<uint64_t*>(a.workspace);
  float2* sums = reinterpret_cast<float2*>(static_cast<char*>(a.workspace) +
                                           align256(size_t(rows * splits * a.num) * 8));
  const RowsK k{a.logits, a.v, a.ldl, uint32_t(splits), int(a.num), keys, sums};
  hipError_t e;
  switch (a.dtype) {
    case kBF16: e = run_rows<Bf16>(k, rows, slice, s); break;
    case kF16: e = run_rows<_Float16>(k, rows, slice, s); break;
    default: e = run_rows<float>(k, rows, slice, s);
  }
  if (e != hipSuccess) return e;
  const PickK p{a.scores,     a.finished,      keys,          sums,           splits,
                int(a.beams), int(a.num),      a.eos,         a.ignore_index, a.scores_out,
                a.parents_out, a.tokens_out,   a.finished_out, a.status_out};
  // within 64 KiB of LDS: 65300 bytes at 64 beams and candidates
  const int waves = int(std::min<int64_t>(a.beams, a.beams * a.num <= 2048 ? 8 : 4));
  const size_t lds = size_t(a.beams * a.num) * 12 + size_t(waves) * (kRowList + kMost) * 8 +
                     size_t(waves) * 4 + 4;
  TimedLaunch t(s, K_BEAM_PICK);
  hipLaunchKernelGGL(beam_pick_kernel, dim3(unsigned(a.batch)), dim3(64 * waves), lds, s, p);
  return hipGetLastError();
}

int64_t beam_reorder_groups(const lce_beam_state& st, int64_t batch, int64_t beams, int64_t slots,
                            bool inplace) {
  const int64_t chunk = inplace ? kTile / beams / 16 * 16 : kChunk;
  const int64_t chunks = (st.segment_bytes + chunk - 1) / chunk;
  return batch * (inplace ? 1 : slots) * st.segments * chunks;
}

hipError_t beam_reorder_run(const lce_beam_state* states, int64_t count, const int32_t* parents,
                            int64_t batch, int64_t beams, int64_t slots, bool inplace,
                            hipStream_t s) {
  for (int64_t at = 0; at < count;) {
    StatesK k{};
    k.parents = parents;
    k.beams = beams;
    k.slots = slots;
    k.chunk = inplace ? kTile / beams / 16 * 16 : kChunk;
    int64_t groups = 0;
    while (at < count && k.count < kStates) {
      const lce_beam_state& st = states[at];
      const int64_t g = beam_reorder_groups(st, batch, beams, slots, inplace);
      if (k.count > 0 && groups + g > (int64_t(1) << 23)) break;  // a launch's threads
      ++at;
      if (g == 0) continue;
      k.st[k.count] = st;
      k.first[k.count] = groups;
      k.chunks[k.count] = (st.segment_bytes + k.chunk - 1) / k.chunk;
      groups += g;
      k.first[++k.count] = groups;
    }
    if (groups == 0) continue;
    TimedLaunch t(s, K_BEAM_REORDER);
    if (inplace)
      hipLaunchKernelGGL(beam_inplace_kernel, dim3(unsigned(groups)), dim3(kThreads), 0, s, k);
    else
      hipLaunchKernelGGL(beam_copy_kernel, dim3(unsigned(groups)), dim3(kThreads), 0, s, k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace lce
