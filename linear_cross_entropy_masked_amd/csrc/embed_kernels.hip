// Embedding lookup with scaling and its gradient, for gfx950.
//
//   lookup    out[i, :] = scale · W[t_i, :]        (0 for a row whose token is ignored or bad)
//   gradient  dW[v, :] (=|+=) scale · Σ_{i: t_i = v} g[i, :]
//
// Both are memory-bound: the lookup reads and writes n rows, the gradient reads n rows and, when
// it overwrites dW, writes all v of them. Every multiply and sum is fp32, rounded once on the
// way out, and a token's rows are added in increasing position without atomics, so a result
// does not change from run to run.
//
// The gradient puts the positions in the order of their tokens first (stable), then walks the
// sorted list in chunks of equal length, so that a token that fills half the batch costs no
// more than the same number of rare ones:
//   1. rank_sort_kernel: runs of kRun positions, each sorted by counting for every key the keys
//      of its run below it. The same launch zeroes the first rows of an overwritten dW, as many
//      as memory takes while the sort computes;
//   2. merge_runs_kernel: up to kMergeWays sorted runs become one per launch, every element
//      finding its place by binary searches (none for n <= kRun);
//   3. segment_sums_kernel: one chunk of sorted positions and one block of columns per thread
//      group; a token wholly inside a chunk is finished there, one that crosses a chunk border
//      leaves a partial sum per chunk. The same launch zeroes the other rows that no position
//      names;
//   4. join_chunks_kernel: the partial sums of each crossing token, added in a fixed order.
// 32768 rows of 4096 bf16 into a bf16 [128256, 4096] table take 306 us: 14 + 17 for the order,
// 262 for the sums (1.3 GB, 4.9 TB/s, the rate of a copy), 16 for the join. Zeroing all of dW in
// the first launch instead took 387: what it leaves in the caches has to be written back while
// the sums read.
#include <algorithm>

#include "common.h"
#include "elem.h"
#include "ops.h"

namespace lce {

namespace {

// Positions per sorted run: ranking costs kRun compares a position, merging one launch where there
// is more than one run (2048 / 4096 / 8192: 316 / 317 / 328 us for 32768 rows as above).
constexpr int kRun = 2048;
constexpr int kFillRows = 16;    // vocabulary rows per zeroing workgroup of the sums
constexpr int kRankWaves = 16;   // wavefronts that share one ranking workgroup's keys
constexpr int kRankLane = 2;                 // positions that one lane ranks
constexpr int kRankRows = 64 * kRankLane;     // and a workgroup
constexpr int kMergeWays = 16;
constexpr int kThreads = 256;

__device__ __forceinline__ bool token_ok(int32_t t, int64_t v, int32_t ignore_index) {
  return t != ignore_index && t >= 0 && int64_t(t) < v;
}

// ------------------------------------------------------------------ lookup

// tpr lanes (a power of two) per row, kVecs vectors each; 256 / tpr rows per workgroup.
constexpr int kLookupVecs = 4;
template <class T>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(
    const T* __restrict__ w, int64_t v, int64_t h, int64_t ldw,
    const int32_t* __restrict__ tokens, int64_t n, int32_t ignore_index, float scale,
    T* __restrict__ out, int64_t ldo, int tpr, int64_t colblocks) {
  constexpr int VE = Elem<T>::kVec;
  const int64_t rb = int64_t(blockIdx.x) / colblocks, cb = int64_t(blockIdx.x) % colblocks;
  const int64_t i = rb * (kThreads / tpr) + threadIdx.x / tpr;
  if (i >= n) return;
  const int32_t t = tokens[i];
  const bool ok = token_ok(t, v, ignore_index);
  const T* src = w + (ok ? int64_t(t) : 0) * ldw;
  T* dst = out + i * ldo;
  const int64_t c0 = (cb * tpr * kLookupVecs + threadIdx.x % tpr) * VE;
  float x[kLookupVecs][VE];
#pragma unroll
  for (int k = 0; k < kLookupVecs; ++k) {
    const int64_t c = c0 + int64_t(k) * tpr * VE;
    if (c < h) load_some<T, VE>(src + c, h - c, x[k]);
  }
#pragma unroll
  for (int k = 0; k < kLookupVecs; ++k) {
    const int64_t c = c0 + int64_t(k) * tpr * VE;
    if (c >= h) continue;
#pragma unroll
    for (int q = 0; q < VE; ++q) x[k][q] = ok ? x[k][q] * scale : 0.f;
    store_some<T, VE>(dst + c, h - c, x[k]);
  }
}

// One workgroup: *status = LCE_STATUS_BAD_TOKEN if some token is neither ignored nor in [0, v).
__global__ void __launch_bounds__(1024) token_status_kernel(const int32_t* __restrict__ tokens,
                                                            int64_t n, int64_t v,
                                                            int32_t ignore_index,
                                                            int32_t* __restrict__ status) {
  __shared__ int any;
  if (threadIdx.x == 0) any = 0;
  __syncthreads();
  int bad = 0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) {
    const int32_t t = tokens[i];
    bad |= int(t != ignore_index && !token_ok(t, v, ignore_index));
  }
  if (bad) any = 1;  // every writer writes the same value
  __syncthreads();
  if (threadIdx.x == 0) *status = any ? LCE_STATUS_BAD_TOKEN : 0;
}

// ------------------------------------------------------------------ sort by token

// One run of kRun positions: position i's key is token · kRun + (i − run start), tokens that
// carry no row counting as v, so keys are distinct and their order is the stable order by
// token. A key's place is the number of keys below it. Workgroup b of a run places kRankRows of its
// positions: kRankWaves wavefronts each count over one slice of the run's keys in LDS. Key is
// uint32_t where (v + 1) · kRun fits, else uint64_t: the compare is most of the work.
//
// Workgroups from sort_blocks on zero a part of dW's first rows each.
struct ZeroArgs {
  void* p;
  int64_t rows, cols, ld;  // one row of all elements where dW is contiguous
};
constexpr int64_t kZeroFirst = int64_t(64) << 20;  // bytes
constexpr int kZeroThreads = 64 * kRankWaves, kZeroVecs = 4;
template <class TW>
__device__ __forceinline__ void zero_part(const ZeroArgs& a, int64_t block) {
  constexpr int VW = Elem<TW>::kVec;
  const int64_t vpr = (a.cols + VW - 1) / VW;
  const float zero[VW] = {};
#pragma unroll
  for (int k = 0; k < kZeroVecs; ++k) {
    const int64_t i = (block * kZeroVecs + k) * kZeroThreads + threadIdx.x;
    const int64_t r = a.rows == 1 ? 0 : i / vpr;
    const int64_t c = (i - r * vpr) * VW;
    if (r < a.rows && c < a.cols)
      store_some<TW, VW>(static_cast<TW*>(a.p) + r * a.ld + c, a.cols - c, zero);
  }
}
template <class TW>
int64_t zero_blocks(const ZeroArgs& a) {
  const int64_t vecs = a.rows * ((a.cols + Elem<TW>::kVec - 1) / Elem<TW>::kVec);
  return (vecs + kZeroThreads * kZeroVecs - 1) / (kZeroThreads * kZeroVecs);
}

template <class Key, class TW>
__global__ void __launch_bounds__(64 * kRankWaves) rank_sort_kernel(
    const int32_t* __restrict__ tokens, int64_t n, int64_t v, int32_t ignore_index,
    int32_t* __restrict__ stok, int32_t* __restrict__ spos, int64_t sort_blocks, ZeroArgs zero) {
  if (int64_t(blockIdx.x) >= sort_blocks) {
    zero_part<TW>(zero, int64_t(blockIdx.x) - sort_blocks);
    return;
  }
  constexpr int kPer = 16 / sizeof(Key);  // keys of one 16-byte LDS read
  __shared__ __attribute__((aligned(16))) Key k[kRun];
  __shared__ int cnt[kRankWaves][kRankRows];
  const int64_t run0 = int64_t(blockIdx.x) / (kRun / kRankRows) * kRun;
  const int64_t left = n - run0;
  const int rows = left < kRun ? int(left) : kRun;
  const int i0 = int(blockIdx.x % (kRun / kRankRows)) * kRankRows;
  if (i0 >= rows) return;  // uniform over the workgroup
  const int padded = (rows + kPer - 1) / kPer * kPer;
  for (int i = threadIdx.x; i < padded; i += 64 * kRankWaves) {
    Key key = ~Key(0);  // padding: below nothing
    if (i < rows) {
      const int32_t t = tokens[run0 + i];
      key = Key(token_ok(t, v, ignore_index) ? int64_t(t) : v) * kRun + Key(i);
    }
    k[i] = key;
  }
  __syncthreads();
  const int r = threadIdx.x & 63, q = threadIdx.x >> 6;
  Key x[kRankLane];
  int below[kRankLane];
#pragma unroll
  for (int u = 0; u < kRankLane; ++u) {
    const int i = i0 + 64 * u + r;
    x[u] = i < rows ? k[i] : Key(0);
    below[u] = 0;
  }
  const int groups = padded / kPer;
  const int per = (groups + kRankWaves - 1) / kRankWaves;
  const int lo = q * per, hi = lo + per < groups ? lo + per : groups;
  struct alignas(16) Pack {
    Key e[kPer];
  };
  const Pack* p = reinterpret_cast<const Pack*>(k);
#pragma unroll 4
  for (int g = lo; g < hi; ++g) {
    const Pack c = p[g];
#pragma unroll
    for (int e = 0; e < kPer; ++e)
#pragma unroll
      for (int u = 0; u < kRankLane; ++u) below[u] += int(c.e[e] < x[u]);
  }
#pragma unroll
  for (int u = 0; u < kRankLane; ++u) cnt[q][64 * u + r] = below[u];
  __syncthreads();
  const int i = i0 + threadIdx.x;
  if (threadIdx.x < kRankRows && i < rows) {
    int place = 0;
#pragma unroll
    for (int w = 0; w < kRankWaves; ++w) place += cnt[w][threadIdx.x];
    stok[run0 + place] = int32_t(k[i] / kRun);
    spos[run0 + place] = int32_t(run0 + i);
  }
}

// Sorted runs of `len` elements (a power of two), kMergeWays at a time into one: an element's
// place is its own index plus, for every other run of its group, the number of elements that come
// before it there (equal tokens of an earlier run do, those of a later run do not). The searches
// of all runs take their steps together: one step's loads do not wait for each other.
constexpr int kMergeThreads = 64;
__global__ void __launch_bounds__(kMergeThreads) merge_runs_kernel(
    const int32_t* __restrict__ tok_in, const int32_t* __restrict__ pos_in,
    int32_t* __restrict__ tok_out, int32_t* __restrict__ pos_out, int64_t n, int64_t len) {
  const int64_t e = int64_t(blockIdx.x) * kMergeThreads + threadIdx.x;
  if (e >= n) return;
  const int32_t t = tok_in[e];
  const int64_t run = e / len, first = run / kMergeWays * kMergeWays;
  const int own = int(run - first);
  int64_t before[kMergeWays];  // elements of each run known to come before
#pragma unroll
  for (int o = 0; o < kMergeWays; ++o) before[o] = 0;
  for (int64_t step = len; step >= 1; step >>= 1) {
    int32_t x[kMergeWays];
    bool in[kMergeWays];
#pragma unroll
    for (int o = 0; o < kMergeWays; ++o) {
      // the last of the run's next `step` elements
      const int64_t at = (first + o) * len + before[o] + step - 1;
      in[o] = o != own && before[o] + step <= len && at < n;
      x[o] = tok_in[in[o] ? at : e];
    }
#pragma unroll
    for (int o = 0; o < kMergeWays; ++o)
      if (in[o] && (x[o] < t || (x[o] == t && o < own))) before[o] += step;
  }
  int64_t place = first * len + (e - run * len);
#pragma unroll
  for (int o = 0; o < kMergeWays; ++o) place += before[o];
  tok_out[place] = t;
  pos_out[place] = pos_in[e];
}

// ------------------------------------------------------------------ sums over equal tokens

struct SegArgs {
  const void* grad;
  int64_t ldg;
  const int32_t* stok;
  const int32_t* spos;
  int64_t n, h, v;
  float scale;
  void* dw;
  int64_t ldw;
  float* part;       // [chunks][2][h] partial sums of the tokens that cross a chunk border
  int64_t len;       // positions per chunk
  int64_t chunks, colblocks, seg_blocks;
  int64_t join_blocks;  // column blocks of the join
  int64_t fill_from;  // rows from here on that no position names are zeroed by the sums' launch
  int tpr;           // lanes per chunk and column block (a power of two)
  const float* coef;       // COEF: row i counts coef[i] times
  const float* scale_dev;  // in place of scale (NULL: not)
  uint32_t* named;         // COEF: the bits of the tokens that have rows are set (NULL: not)
  __device__ __forceinline__ float factor() const { return scale_dev ? *scale_dev : scale; }
};

// The first index in [0, n) whose token is >= t, found by the 64 lanes of a wavefront together:
// each step probes 64 places, so n = 2^18 takes three dependent loads instead of eighteen.
__device__ __forceinline__ int64_t wave_lower_bound(const int32_t* __restrict__ stok, int64_t n,
                                                    int32_t t) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t step = (hi - lo + 63) >> 6;
    const int64_t p = lo + (lane + 1) * step - 1;
    const bool less = p < hi && stok[p] < t;
    const int64_t c = __popcll(__ballot(less));
    lo += c * step;
    const int64_t h2 = lo + step - 1;
    if (h2 < hi) hi = h2;
  }
  return lo;
}

// A finished sum as it goes into the table. Weighted ones are rounded to bf16 whatever the table's
// type, so that what is built on them is the same in both: for flce_pieces.hip half a step of a
// remainder of half a step.
template <bool COEF>
__device__ __forceinline__ float finished(float scale, float acc) {
  return scale * (COEF ? bf16_to_f32(f32_to_bf16(acc)) : acc);
}
template <class TW, int N, bool ACC, bool COEF>
__device__ __forceinline__ void put_sum(TW* p, int64_t cnt, float scale, const float (&acc)[N]) {
  float x[N];
  if constexpr (ACC) {
    load_some<TW, N>(p, cnt, x);
#pragma unroll
    for (int q = 0; q < N; ++q) x[q] += finished<COEF>(scale, acc[q]);
  } else {
#pragma unroll
    for (int q = 0; q < N; ++q) x[q] = finished<COEF>(scale, acc[q]);
  }
  store_some<TW, N>(p, cnt, x);
}

constexpr int kBatch = 4;  // rows in flight per lane (8: 314 us, 16: 374 us where 4 take 306)

template <class T, class TW, bool ACC, bool COEF>
__global__ void __launch_bounds__(kThreads) segment_sums_kernel(SegArgs a) {
  constexpr int VE = Elem<T>::kVec;
  TW* const dw = static_cast<TW*>(a.dw);
  const int64_t bx = blockIdx.x;
  if (bx >= a.seg_blocks) {
    // rows that no position names, four per wavefront
    if constexpr (!ACC) {
      constexpr int kRows = kFillRows / (kThreads / 64);
      const int lane = threadIdx.x & 63;
      const int64_t r0 = a.fill_from + (bx - a.seg_blocks) * kFillRows +
                         int64_t(threadIdx.x >> 6) * kRows;
      bool named[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int64_t p = wave_lower_bound(a.stok, a.n, int32_t(r0 + k));
        named[k] = r0 + k >= a.v || (p < a.n && a.stok[p] == int32_t(r0 + k));
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (named[k]) continue;
        constexpr int VW = Elem<TW>::kVec;
        const float zero[VW] = {};
        for (int64_t c = int64_t(lane) * VW; c < a.h; c += 64 * VW) {
          if (a.h - c >= VW) {  // never read here again: past the caches (343 us so, 367 without)
            store_stream(dw + (r0 + k) * a.ldw + c, Elem<TW>::pack(zero));
            continue;
          }
          store_some<TW, VW>(dw + (r0 + k) * a.ldw + c, a.h - c, zero);
        }
      }
    }
    return;
  }
  const int64_t item = bx * (kThreads / a.tpr) + threadIdx.x / a.tpr;
  const int64_t chunk = item / a.colblocks, cb = item % a.colblocks;
  if (chunk >= a.chunks) return;
  const int64_t col = (cb * a.tpr + threadIdx.x % a.tpr) * VE;
  if (col >= a.h) return;
  const int64_t cnt = a.h - col;
  const T* const g = static_cast<const T*>(a.grad) + col;
  const int64_t p0 = chunk * a.len;
  const int64_t p1 = p0 + a.len < a.n ? p0 + a.len : a.n;
  const int32_t none = int32_t(a.v);  // sorted after every token: positions without a row
  int32_t cur = a.stok[p0];
  if (cur >= none) return;
  bool from_left = p0 > 0 && a.stok[p0 - 1] == cur;
  const float scale = a.factor();
  float acc[VE] = {};
  auto flush = [&](bool to_right) {
    if (COEF && a.named && col == 0) atomicOr(a.named + (cur >> 5), 1u << (cur & 31));
    if (from_left || to_right) {
      float* p = a.part + (chunk * 2 + (from_left ? 0 : 1)) * a.h + col;
#pragma unroll
      for (int q = 0; q < VE; ++q)
        if (q < cnt) p[q] = acc[q];
    } else {
      put_sum<TW, VE, ACC, COEF>(dw + int64_t(cur) * a.ldw + col, cnt, scale, acc);
    }
  };
  for (int64_t p = p0; p < p1; p += kBatch) {
    int32_t tok[kBatch];
    float x[kBatch][VE], c[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      tok[u] = p + u < p1 ? a.stok[p + u] : none;
      const int64_t row = tok[u] < none ? a.spos[p + u] : 0;
      if (tok[u] < none) load_some<T, VE>(g + row * a.ldg, cnt, x[u]);
      c[u] = COEF && tok[u] < none ? a.coef[row] : 1.f;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (tok[u] >= none) break;
      if (tok[u] != cur) {
        flush(false);
        cur = tok[u];
        from_left = false;
#pragma unroll
        for (int q = 0; q < VE; ++q) acc[q] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < VE; ++q) acc[q] += COEF ? c[u] * x[u][q] : x[u][q];
    }
  }
  flush(p1 < a.n && a.stok[p1] == cur);
}

// The token that starts in a chunk and runs past its end: its partial sums, in chunk order within
// a wavefront (every fourth chunk) and then in wavefront order. Four columns a lane, 256 a
// workgroup; the token's end is searched for, so that the loads do not wait for one another.
constexpr int kJoinCols = 256;
template <class T, class TW, bool ACC, bool COEF>
__global__ void __launch_bounds__(256) join_chunks_kernel(SegArgs a) {
  const int64_t chunk = int64_t(blockIdx.x) / a.join_blocks;
  const int64_t p0 = chunk * a.len, p1 = p0 + a.len;  // a later chunk exists: p1 < n
  const int32_t cur = a.stok[p1 - 1], after = a.stok[p1], before = a.stok[p0 > 0 ? p0 - 1 : 0];
  if (cur >= int32_t(a.v) || after != cur) return;
  if (p0 > 0 && before == cur) return;  // it starts in an earlier chunk
  const int64_t end = p1 + wave_lower_bound(a.stok + p1, a.n - p1, cur + 1);
  const int64_t last = (end - 1) / a.len;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = int64_t(blockIdx.x) % a.join_blocks * kJoinCols + 4 * lane;
  const int64_t cnt = a.h - col;
  float acc[4] = {};
  if (cnt > 0) {
    if (wave == 0) load_some<float, 4>(a.part + (chunk * 2 + 1) * a.h + col, cnt, acc);
    int64_t c = chunk + 1 + wave;
    for (; c + 4 * (kBatch - 1) <= last; c += 4 * kBatch) {
      float x[kBatch][4];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        load_some<float, 4>(a.part + (c + 4 * u) * 2 * a.h + col, cnt, x[u]);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] += x[u][q];
    }
    for (; c <= last; c += 4) {
      float x[4];
      load_some<float, 4>(a.part + c * 2 * a.h + col, cnt, x);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] += x[q];
    }
  }
  __shared__ float sum[4][kJoinCols];
#pragma unroll
  for (int q = 0; q < 4; ++q) sum[wave][4 * lane + q] = acc[q];
  __syncthreads();
  if (wave != 0 || cnt <= 0) return;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    acc[q] = ((sum[0][4 * lane + q] + sum[1][4 * lane + q]) + sum[2][4 * lane + q]) +
             sum[3][4 * lane + q];
  const float scale = a.factor();
  TW* d = static_cast<TW*>(a.dw) + int64_t(cur) * a.ldw + col;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q >= cnt) break;
    const float x = finished<COEF>(scale, acc[q]);
    d[q] = Elem<TW>::from_f32(ACC ? Elem<TW>::to_f32(d[q]) + x : x);
  }
}

int pow2_at_least(int64_t x, int cap) {
  int p = 1;
  while (p < cap && p < x) p <<= 1;
  return p;
}

// Positions per chunk: about 1024 chunks, at least 8 positions (the rows one lane has in
// flight) and at most 512 (so that the partial sums of one chunk border stay a small share of
// the rows read). Weighted rows take about 512 chunks: half the partial sums, which stand beside the
// logit gradients there.
constexpr int64_t kChunks = 1024, kWeightedChunks = 512;
int64_t chunk_len(int64_t n, int64_t most) {
  return pow2_at_least(std::max<int64_t>(8, (n + most - 1) / most), 512);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct EmbedWs {
  int32_t *tok[2], *pos[2];
  float* part;
  size_t bytes;
};
EmbedWs carve(void* base, int64_t n, int64_t h, int64_t most) {
  char* b = static_cast<char*>(base);
  EmbedWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = b + off;
    off += align256(bytes);
    return p;
  };
  const int bufs = n > kRun ? 2 : 1;
  for (int k = 0; k < bufs; ++k) {
    w.tok[k] = reinterpret_cast<int32_t*>(take(size_t(n) * 4));
    w.pos[k] = reinterpret_cast<int32_t*>(take(size_t(n) * 4));
  }
  const int64_t len = chunk_len(n, most), chunks = (n + len - 1) / len;
  w.part = reinterpret_cast<float*>(take(size_t(chunks) * 2 * size_t(h) * 4));
  w.bytes = std::max<size_t>(off, 256);
  return w;
}

template <class T, class TW, bool ACC, bool COEF>
hipError_t run_segments(const SegArgs& a, hipStream_t s) {
  {
    TimedLaunch t(s, K_EMBED_GRAD);
    const int64_t fill = ACC || COEF ? 0 : (a.v - a.fill_from + kFillRows - 1) / kFillRows;
    hipLaunchKernelGGL((segment_sums_kernel<T, TW, ACC, COEF>), dim3(unsigned(a.seg_blocks + fill)),
                       dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.chunks <= 1) return e;
  }
  TimedLaunch t(s, K_EMBED_JOIN);
  hipLaunchKernelGGL((join_chunks_kernel<T, TW, ACC, COEF>),
                     dim3(unsigned((a.chunks - 1) * a.join_blocks)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <class T, class TW, bool COEF = false>
hipError_t run_bwd(const EmbedBwdArgs& a, hipStream_t s, const float* coef = nullptr,
                   const float* scale_dev = nullptr, bool sorted = false,
                   uint32_t* named = nullptr) {
  constexpr int64_t kMost = COEF ? kWeightedChunks : kChunks;
  const bool acc = (a.flags & EMBED_ACCUMULATE) != 0, keep = acc || COEF;
  const EmbedWs ws = carve(a.workspace, a.n, a.h, kMost);
  const int64_t runs = (a.n + kRun - 1) / kRun;
  const int64_t last = a.n - (runs - 1) * kRun;
  const int64_t sort_blocks =
      a.n > 0 ? (runs - 1) * (kRun / kRankRows) + (last + kRankRows - 1) / kRankRows : 0;
  // without positions there is no launch of the sums: all of dW at once
  const int64_t most = kZeroFirst / (a.h * int64_t(sizeof(TW)));
  const int64_t first = keep ? 0 : a.n == 0 ? a.v : std::min(a.v, most);
  ZeroArgs zero{a.grad_weight, first, a.h, a.ldw};
  if (a.ldw == a.h) zero = ZeroArgs{a.grad_weight, 1, first * a.h, 0};
  const int64_t blocks = sort_blocks + (keep ? 0 : zero_blocks<TW>(zero));
  hipError_t e;
  if (blocks > 0 && !sorted) {
    TimedLaunch t(s, K_EMBED_SORT);
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(unsigned(blocks)), dim3(64 * kRankWaves), 0, s, a.tokens,
                         a.n, a.v, a.ignore_index, ws.tok[0], ws.pos[0], sort_blocks, zero);
    };
    if (a.v + 1 <= int64_t(0xffffffffLL) / kRun)
      launch(rank_sort_kernel<uint32_t, TW>);
    else
      launch(rank_sort_kernel<uint64_t, TW>);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.n == 0) return hipSuccess;
  int cur = 0;
  for (int64_t len = kRun; len < a.n && !sorted; len *= kMergeWays) {
    TimedLaunch t(s, K_EMBED_SORT);
    hipLaunchKernelGGL(merge_runs_kernel,
                       dim3(unsigned((a.n + kMergeThreads - 1) / kMergeThreads)),
                       dim3(kMergeThreads), 0, s, ws.tok[cur], ws.pos[cur], ws.tok[cur ^ 1],
                       ws.pos[cur ^ 1], a.n, len);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    cur ^= 1;
  }
  SegArgs g{};
  g.grad = a.grad;
  g.ldg = a.ldg;
  g.stok = ws.tok[cur];
  g.spos = ws.pos[cur];
  g.n = a.n;
  g.h = a.h;
  g.v = a.v;
  g.scale = a.scale;
  g.dw = a.grad_weight;
  g.ldw = a.ldw;
  g.part = ws.part;
  g.join_blocks = (a.h + kJoinCols - 1) / kJoinCols;
  g.fill_from = first;
  g.len = chunk_len(a.n, kMost);
  g.chunks = (a.n + g.len - 1) / g.len;
  const int64_t vecs = (a.h + Elem<T>::kVec - 1) / Elem<T>::kVec;
  g.tpr = pow2_at_least(vecs, kThreads);
  g.colblocks = (vecs + g.tpr - 1) / g.tpr;
  const int64_t per = kThreads / g.tpr;
  g.seg_blocks = (g.chunks * g.colblocks + per - 1) / per;
  g.coef = coef;
  g.scale_dev = scale_dev;
  g.named = named;
  return acc ? run_segments<T, TW, true, COEF>(g, s) : run_segments<T, TW, false, COEF>(g, s);
}

template <class T>
hipError_t run_lookup(const EmbedFwdArgs& a, hipStream_t s) {
  constexpr int VE = Elem<T>::kVec;
  const int64_t vecs = (a.h + VE - 1) / VE;
  const int tpr = pow2_at_least((vecs + kLookupVecs - 1) / kLookupVecs, kThreads);
  const int64_t colblocks = (vecs + int64_t(tpr) * kLookupVecs - 1) / (int64_t(tpr) * kLookupVecs);
  const int64_t rpw = kThreads / tpr, blocks = (a.n + rpw - 1) / rpw * colblocks;
  TimedLaunch t(s, K_EMBED_FWD);
  hipLaunchKernelGGL((embed_fwd_kernel<T>), dim3(unsigned(blocks)), dim3(kThreads), 0, s,
                     static_cast<const T*>(a.weight), a.v, a.h, a.ldw, a.tokens, a.n,
                     a.ignore_index, a.scale, static_cast<T*>(a.out), a.ldo, tpr, colblocks);
  return hipGetLastError();
}

hipError_t token_status(const int32_t* tokens, int64_t n, int64_t v, int32_t ignore_index,
                        int32_t* status, hipStream_t s) {
  if (!status) return hipSuccess;
  TimedLaunch t(s, K_LABEL_PREP);
  hipLaunchKernelGGL(token_status_kernel, dim3(1), dim3(1024), 0, s, tokens, n, v, ignore_index,
                     status);
  return hipGetLastError();
}

}  // namespace

hipError_t embed_fwd_run(const EmbedFwdArgs& a, hipStream_t s) {
  hipError_t e = token_status(a.tokens, a.n, a.v, a.ignore_index, a.status_out, s);
  if (e != hipSuccess || a.n == 0) return e;
  switch (a.dtype) {
    case kBF16: return run_lookup<Bf16>(a, s);
    case kF16: return run_lookup<_Float16>(a, s);
    default: return run_lookup<float>(a, s);
  }
}

size_t embed_workspace_bytes(int64_t n, int64_t h) {
  return carve(nullptr, n, h, kChunks).bytes;
}
size_t embed_weighted_workspace_bytes(int64_t n, int64_t h) {
  return carve(nullptr, n, h, kWeightedChunks).bytes;
}

hipError_t embed_bwd_run(const EmbedBwdArgs& a, hipStream_t s) {
  hipError_t e = token_status(a.tokens, a.n, a.v, a.ignore_index, a.status_out, s);
  if (e != hipSuccess) return e;
  const bool wide = a.grad_dtype == kF32;
  switch (a.dtype) {
    case kBF16: return wide ? run_bwd<Bf16, float>(a, s) : run_bwd<Bf16, Bf16>(a, s);
    case kF16: return wide ? run_bwd<_Float16, float>(a, s) : run_bwd<_Float16, _Float16>(a, s);
    default: return run_bwd<float, float>(a, s);
  }
}

void embed_weighted_order(void* workspace, int64_t n, int64_t h, int32_t** tokens, int32_t** rows) {
  const EmbedWs w = carve(workspace, n, h, kWeightedChunks);
  *tokens = w.tok[0];
  *rows = w.pos[0];
}

hipError_t embed_weighted_run(const EmbedBwdArgs& a, const float* coef, const float* scale,
                              bool sorted, uint32_t* named, hipStream_t s) {
  return a.grad_dtype == kF32 ? run_bwd<Bf16, float, true>(a, s, coef, scale, sorted, named)
                              : run_bwd<Bf16, Bf16, true>(a, s, coef, scale, sorted, named);
}

}  // namespace lce
