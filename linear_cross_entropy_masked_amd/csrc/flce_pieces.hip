// Linear cross entropy taken in pieces of the vocabulary, for gfx950.
//
// z = hidden · Wᵀ + b over a piece W of consecutive vocabulary rows; per row the state
// (max, Σ exp(z − max), label logit) is carried from piece to piece, so neither the logits nor
// anything else of the vocabulary's size is kept. The backward takes each piece by itself:
//   D = c_i · (exp(z − lse) − [v = y])      logits recomputed, bf16, the piece's only big buffer
//   dH (+)= s · D · W                       fp32 over the pieces, bf16 after the last
//   dW  =   s · Dᵀ · hidden                 finished: a piece sees every row
//   db  =   s · Σ_i D                       from the fp32 values
// with s = g / T and c_i = 1 (summed loss), or s the largest of the rows' own upstream gradients
// and c_i the row's share of it.
// Four products of 2 · N · H · V flop in all, on the MFMA tile of gemm_tile.h, and bound by them:
// 8192 x 4096 x 128256, 5% of the rows without a label, takes 6.5 ms forward and 20 ms backward
// (logits 7.0, dH 6.5, dW 6.5; 1.17 to 1.27 PFLOP/s).
//
// Rows without a label are left out of every product: the labelled rows are numbered, their hidden
// rows copied together (gather_few_rows_kernel, or piece_rows_kernel and gather_rows_kernel for
// long batches), and the products stop at the count that leaves in device memory. That also keeps
// whatever such rows hold (NaN in a padded position) out of dW. The copy costs 4 · N · H bytes
// against 2 · N · H · V flop.
//
// D is rounded to bf16 (an MFMA operand) once, without the factor s, so that the rounding is
// independent from element to element: a common factor would be rounded the same way in every
// label element, and scale both gradients with it (by 1.0025 for rows that all have 1 / 1003).
// Half a bf16 step per element. A row's label element is as large as all its others together, and
// what the rounding leaves of it is kept in fp32 (e_i) and added to the products: s · e_i · W[y_i] to
// dH, s · e_i · hidden_i to row y_i of dW, the rows put in the order of their labels as for the
// table's gradient (embed_kernels.hip; a bf16 dW that is added to has no bits for that). 1024 rows of
// 768 and 32777 classes, label logits raised by 0 / 6 / 12: norm-wise error of dW in fp32 2.8e-5 /
// 2.9e-5 / 3.1e-5, and 6.4e-5 / 1.1e-3 / 1.6e-3 without the remainder; of dW in bf16 1.47e-3 / 1.65e-3
// / 1.66e-3, its own rounding, and 1.47e-3 / 1.99e-3 / 2.28e-3. It takes 14 to 22 us a piece (the
// order in the gather, two launches for the sums, the products' start), 20 of 376 us of the step of
// 2048 x 768 x 32777 with half the rows labelled, 0.2 to 0.4 of 27 ms at 8192 x 4096 x 128256. Step
// times that compare two forms below are without it on either side.
//
// With at most kScoreRows rows the forward is bound by reading W once, and score_kernel streams
// it past the rows instead; up to kNarrowRows rows take tiles of half the height with three K
// slices in the ring, and products of few tiles smaller ones.
#include <algorithm>

#include "common.h"
#include "flce_pieces.h"
#include "gemm_tile.h"
#include "lce_masked.h"
#include "ops.h"

namespace lce {

namespace {

using gemm::View;
using gemm::f32x4_t;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
using Wide = gemm::v2::CfgWide;
using Pair = gemm::v2::CfgPair;
using Narrow = gemm::v2::Cfg<128, 256, 64, 3, 2, 4, 1>;
using Small = gemm::v2::Cfg<128, 128, 64, 4, 2, 2, 1>;

__host__ __device__ inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Tile order of the two logits products: bands of 8 row tiles, so that the 32 tiles in flight on
// an XCD read 8 + 4 tiles of operands instead of 31 + 1 (8192 x 4096 x 128256 forward 7.0 -> 6.45
// ms, the whole step 27.5 -> 26.8; bands of 4 and 16 the same). The gradients' products keep the
// block of tiles per XCD (26.9 and 27.2 in bands).
constexpr int kBand = 8;

constexpr int kTile = Wide::BM;  // rows of an output tile; the gathered rows are padded to it
// 32 / 64 rows of 4096 against 128256 classes take 222 / 276 us in the scoring kernel, 32 / 64 / 128
// rows 221 / 223 / 221 on 128 x 256 tiles and 269 / 271 / 267 on 256 x 256 tiles (20 rows: 204,
// 229, 275); 256 rows take 284 us on 256 x 256 tiles and 317 on 128 x 256.
constexpr int kScoreRows = 32;
constexpr int kNarrowRows = 128;
// The weight gradient's contraction is as long as the batch. Where it has a launch of its own, up
// to this many rows it is mostly stores, and two 256 x 128 workgroups per CU overlap them (step of
// 60 rows of 2048 and 60000 classes 306 us against 323, of 500 rows and 32000 classes 338 against
// 344, of 1000 rows of 4096 1005 against 994).
constexpr int kShortK = 512;

// Products whose 128 x 128 tiles all run at once take those, with three K slices in flight: with so
// few tiles a product is a chain of slices, each as long as its loads (steps of 682 rows of 3840 and
// 2066 classes 169 us so and 263 without, 3633 of 88 and 24693 331 and 367, losses of 189 rows of
// 1904 and 2404 classes 43 and 68; twice as many tiles: 500 rows of 1024 and 15000 classes 153, 151
// without).
constexpr int64_t kFewTiles = 256;
bool few_tiles(int64_t m, int64_t n) {
  return (m + Small::BM - 1) / Small::BM * ((n + Small::BN - 1) / Small::BN) <= kFewTiles;
}
// Classes per tile of the forward's logits product, rows per tile of the backward's.
int64_t lse_cols(int64_t n, int64_t v) { return few_tiles(n, v) ? Small::BN : Wide::BN; }
int grad_rows(int64_t n, int64_t v) {
  return few_tiles(n, v) || n <= kNarrowRows ? Small::BM : Wide::BM;
}

__device__ __forceinline__ bool labelled(int32_t y, int64_t vocab, int32_t ignore_index) {
  return y != ignore_index && y >= 0 && int64_t(y) < vocab;
}

// Where the kernel that counts the labelled rows leaves s = g / T (0 when T = 0). out is NULL where
// no s is asked for, or where row_scale_kernel has written it.
struct ScaleOut {
  float* out;
  long long t_host;
  const float* gout;
  __device__ __forceinline__ void put(long long count) const {
    if (!out) return;
    const long long t = t_host >= 0 ? t_host : count;
    *out = t > 0 ? float(double(gout ? *gout : 1.f) / double(t)) : 0.f;
  }
};

// The least maximum a block's exponentials are taken about: where the bias masks every class of a
// block with minus infinity, there is then a number to subtract, and the sum is 0.
constexpr float kLeastMax = -3.4028234663852886e38f;

// s for per-row upstream gradients, in one workgroup: the largest finite magnitude among the labelled
// rows, 1 where that is 0. The other rows' may be anything; a row whose own is infinite or NaN gets
// that into its gradient, and leaves s to the others.
__global__ void __launch_bounds__(1024) row_scale_kernel(
    const float* __restrict__ grad_rows, const int32_t* __restrict__ labels, int64_t n,
    int64_t vocab, int32_t ignore_index, float* __restrict__ scale) {
  __shared__ float most[16];
  float m = 0.f;
  for (int64_t i = threadIdx.x; i < n; i += 1024) {
    const float c = fabsf(grad_rows[i]);
    if (labelled(labels[i], vocab, ignore_index) && c < INFINITY) m = fmaxf(m, c);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 16; ++w) m = fmaxf(m, most[w]);
  *scale = m > 0.f ? m : 1.f;
}

// ------------------------------------------------------------------ the labelled rows

// Numbers the rows that carry a label in their order: cidx[i] = the row's number or −1, and for
// the m-th of them row[m] = i and ylab[m] = its label relative to the piece (−1 outside it, and up
// to up(n, kTile)); *count of them. With `state`, the other rows' state is set to (−inf, 0, 0). One workgroup,
// kRowsPer rows a thread and round.
constexpr int kRowsPer = 8;
__global__ void __launch_bounds__(1024) piece_rows_kernel(
    const int32_t* __restrict__ labels, int64_t n, int64_t v, int64_t v_start, int64_t vocab,
    int32_t ignore_index, int32_t* __restrict__ count, int32_t* __restrict__ cidx,
    int32_t* __restrict__ row, int32_t* __restrict__ ylab, float* __restrict__ state,
    ScaleOut scale) {
  __shared__ int wave_sum[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int done = 0;
  for (int64_t base = 0; base < n; base += 1024 * kRowsPer) {
    const int64_t i0 = base + int64_t(threadIdx.x) * kRowsPer;
    int32_t y[kRowsPer];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
      y[k] = i0 + k < n ? labels[i0 + k] : ignore_index;
      mine += labelled(y[k], vocab, ignore_index);
    }
    int upto = mine;  // inclusive sum over the wavefront
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(upto, off, 64);
      if (lane >= off) upto += o;
    }
    __syncthreads();  // the last round's sums have been read
    if (lane == 63) wave_sum[wave] = upto;
    __syncthreads();
    int before = done, total = 0;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) before += wave_sum[w];
      total += wave_sum[w];
    }
    int m = before + upto - mine;
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
      const int64_t i = i0 + k;
      if (i >= n) break;
      if (labelled(y[k], vocab, ignore_index)) {
        const int64_t d = int64_t(y[k]) - v_start;
        cidx[i] = m;
        row[m] = int32_t(i);
        ylab[m] = d >= 0 && d < v ? int32_t(d) : -1;
        ++m;
      } else {
        cidx[i] = -1;
        if (state) {
          state[i] = -INFINITY;
          state[n + i] = 0.f;
          state[2 * n + i] = 0.f;
        }
      }
    }
    done += total;
  }
  for (int64_t m = done + int64_t(threadIdx.x); m < up(n, kTile); m += 1024) ylab[m] = -1;
  if (threadIdx.x == 0) {
    *count = done;
    scale.put(done);
  }
}

struct GatherArgs {
  const uint16_t* hidden;
  int64_t n, h, h64;
  int32_t* count;
  int32_t* cidx;
  int32_t* row;
  int32_t* ylab;
  uint16_t* hc;            // [up(n, kTile)][h64]
  // backward only
  uint32_t* named;         // of so many words, cleared here (NULL: not)
  int64_t words;
  int32_t *stok, *spos;    // gather_few_rows_kernel<true>: the rows in the order of ylab
  const float* lse;
  const float* grad_rows;
  const float* row_scale;  // c_i = grad_rows[i] / *row_scale
  ScaleOut scale;
  float* lse_c;
  float* coef_c;
  float* zero_acc;         // rows without a label are zeroed here (NULL: not)
  uint16_t* zero_grad;
};

// Row i of the batch to its place m: its hidden row, zero-padded to h64 columns.
__device__ __forceinline__ void gather_row(const GatherArgs& a, int64_t i, int64_t m) {
  const uint4 zero = {0u, 0u, 0u, 0u};
  for (int64_t c = 8 * int64_t(threadIdx.x); c < a.h64; c += 8 * 256)
    *reinterpret_cast<uint4*>(a.hc + m * a.h64 + c) =
        c < a.h ? *reinterpret_cast<const uint4*>(a.hidden + i * a.h + c) : zero;
  if (threadIdx.x == 0) {
    if (a.lse_c) a.lse_c[m] = a.lse[i];
    if (a.coef_c) a.coef_c[m] = a.grad_rows[i] / *a.row_scale;
  }
}
// The outputs of a row without a label.
__device__ __forceinline__ void clear_row(const GatherArgs& a, int64_t i) {
  const uint4 zero = {0u, 0u, 0u, 0u};
  if (a.zero_acc)
    for (int64_t c = 4 * int64_t(threadIdx.x); c < a.h; c += 4 * 256)
      *reinterpret_cast<uint4*>(a.zero_acc + i * a.h + c) = zero;
  if (a.zero_grad)
    for (int64_t c = 8 * int64_t(threadIdx.x); c < a.h; c += 8 * 256)
      *reinterpret_cast<uint4*>(a.zero_grad + i * a.h + c) = zero;
}
// Row m past the count, up to the next multiple of the tile: one that contributes nothing.
__device__ __forceinline__ void pad_row(const GatherArgs& a, int64_t m, int64_t count) {
  if (m >= up(count, kTile)) return;
  for (int64_t c = 8 * int64_t(threadIdx.x); c < a.h64; c += 8 * 256)
    *reinterpret_cast<uint4*>(a.hc + m * a.h64 + c) = uint4{0u, 0u, 0u, 0u};
  if (threadIdx.x == 0) {
    if (a.lse_c) a.lse_c[m] = INFINITY;
    if (a.coef_c) a.coef_c[m] = 0.f;
  }
}

__device__ __forceinline__ void clear_named(const GatherArgs& a) {
  if (!a.named) return;
  for (int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x; c < a.words;
       c += int64_t(gridDim.x) * 256)
    a.named[c] = 0;
}

// One workgroup per row of the batch, numbered by piece_rows_kernel, then kTile for the padding.
__global__ void __launch_bounds__(256) gather_rows_kernel(GatherArgs a) {
  const int64_t i = blockIdx.x;
  clear_named(a);
  if (i >= a.n) {
    const int64_t count = *a.count;
    pad_row(a, count + (i - a.n), count);
    return;
  }
  const int64_t m = a.cidx[i];
  if (m >= 0)
    gather_row(a, i, m);
  else
    clear_row(a, i);
}

// Numbering and gathering in one launch, for batches short enough that every workgroup can count
// the labelled rows before its own: `each` rows per workgroup (one for the shortest batches, where
// a row's copy is all latency, else kFewEach; a divisor of kTile). ORDER: with the order of the
// labels, for which each workgroup finds its rows' places on the way: the number of rows whose label
// in the piece is smaller, or the same and earlier (labels outside it count as v, after all others).
constexpr int64_t kFewRows = 8192;
constexpr int kFewEach = 4;
int few_each(int64_t n) { return n <= 1024 ? 1 : kFewEach; }
template <bool ORDER>
__global__ void __launch_bounds__(256) gather_few_rows_kernel(
    GatherArgs a, const int32_t* __restrict__ labels, int64_t v, int64_t v_start, int64_t vocab,
    int32_t ignore_index, int each, float* __restrict__ state) {
  const int64_t batch = (a.n + each - 1) / each;
  const bool padding = int64_t(blockIdx.x) >= batch;
  const int64_t i0 = padding ? a.n : int64_t(blockIdx.x) * each;
  clear_named(a);
  auto label_at = [&](int32_t y) {  // its class in the piece
    const int64_t d = int64_t(y) - v_start;
    return labelled(y, vocab, ignore_index) && d >= 0 && d < v ? int32_t(d) : int32_t(v);
  };
  constexpr int kSums = ORDER ? 1 + kFewEach : 1;
  __shared__ int wave_sum[4][kSums];
  int sum[kSums] = {};  // labelled rows before i0, places of the rows from there
  if constexpr (ORDER) {
    int32_t key[kFewEach];
#pragma unroll
    for (int k = 0; k < kFewEach; ++k)
      key[k] = k < each && i0 + k < a.n ? label_at(labels[i0 + k]) : -1;
    for (int64_t j = threadIdx.x; j < a.n; j += 256) {
      const int32_t y = labels[j], t = label_at(y);
      sum[0] += j < i0 && labelled(y, vocab, ignore_index);
#pragma unroll
      for (int k = 0; k < kFewEach; ++k)
        sum[1 + k] += t < key[k] || (t == key[k] && j < i0 + k);
    }
  } else {
    for (int64_t j = threadIdx.x; j < i0; j += 256)
      sum[0] += labelled(labels[j], vocab, ignore_index);
  }
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum[k] += __shfl_xor(sum[k], off, 64);
    if ((threadIdx.x & 63) == 0) wave_sum[threadIdx.x >> 6][k] = sum[k];
  }
  __syncthreads();
  auto total = [&](int k) {
    return (wave_sum[0][k] + wave_sum[1][k]) + (wave_sum[2][k] + wave_sum[3][k]);
  };
  int64_t m = total(0);
  if (padding) {
    if (int64_t(blockIdx.x) == batch) {
      for (int64_t j = m + threadIdx.x; j < up(a.n, kTile); j += 256) a.ylab[j] = -1;
      if (threadIdx.x == 0) {
        *a.count = int32_t(m);
        a.scale.put(m);
      }
    }
    for (int k = 0; k < each; ++k)
      pad_row(a, m + (int64_t(blockIdx.x) - batch) * each + k, m);
    return;
  }
  for (int64_t i = i0; i < i0 + each && i < a.n; ++i) {
    const int32_t y = labels[i];
    if constexpr (ORDER) {
      if (threadIdx.x == 0) {
        const int place = total(1 + int(i - i0));
        a.stok[place] = label_at(y);
        a.spos[place] = int32_t(m);
      }
    }
    if (labelled(y, vocab, ignore_index)) {
      gather_row(a, i, m);
      if (threadIdx.x == 0) {
        const int64_t d = int64_t(y) - v_start;
        a.row[m] = int32_t(i);
        a.ylab[m] = d >= 0 && d < v ? int32_t(d) : -1;
      }
      ++m;
    } else {
      clear_row(a, i);
      if (state && threadIdx.x == 0) {
        state[i] = -INFINITY;
        state[a.n + i] = 0.f;
        state[2 * a.n + i] = 0.f;
      }
    }
  }
}

// W [v, h] to [v, h64], zero-padded (h not a multiple of the K slice).
constexpr int64_t kPadGrid = 65536;
__global__ void __launch_bounds__(256) pad_rows_kernel(const uint16_t* __restrict__ w, int64_t v,
                                                       int64_t h, int64_t h64,
                                                       uint16_t* __restrict__ out) {
  for (int64_t r = blockIdx.x; r < v; r += gridDim.x)
    for (int64_t c = 8 * int64_t(threadIdx.x); c < h64; c += 8 * 256)
      *reinterpret_cast<uint4*>(out + r * h64 + c) =
          c < h ? *reinterpret_cast<const uint4*>(w + r * h + c) : uint4{0u, 0u, 0u, 0u};
}

// ------------------------------------------------------------------ forward

// bias[n .. n + 3], the last class's past the end (those columns are not used).
__device__ __forceinline__ f32x4_t bias4(const float* bias, int64_t n, int64_t v) {
  f32x4_t b{0.f, 0.f, 0.f, 0.f};
  if (bias) {
#pragma unroll
    for (int q = 0; q < 4; ++q) b[q] = bias[n + q < v ? n + q : v - 1];
  }
  return b;
}

// The logits tile reduced to each row's (max, Σ exp(z − max)), and the label's logit.
struct EpiPieceLse {
  static constexpr bool kRowStats = true, kColSums = false, kTileMax = false, kRowTag = true;
  static constexpr bool kRowLimit = true, kColAux = true;
  const float* bias;
  int64_t v;
  const int32_t* ylab;
  const int32_t* count;
  float2* part;
  int64_t tiles;
  float* zy;
  using Col = f32x4_t;
  struct Aux {
    int y;
  };
  __device__ void begin(int64_t) {}
  __device__ __forceinline__ int64_t row_limit() const { return *count; }
  __device__ __forceinline__ int row_tag(int64_t m) const { return ylab[m]; }
  __device__ __forceinline__ Col load_col(int64_t n) const { return bias4(bias, n, v); }
  __device__ __forceinline__ Aux load4t(int64_t, int64_t, int y) const { return {y}; }
  __device__ __forceinline__ f32x4_t value4c(f32x4_t a, Col b) const { return a + b; }
  __device__ __forceinline__ float value1(int64_t n, float a) const {
    return bias ? a + bias[n] : a;
  }
  __device__ __forceinline__ f32x4_t store4c(int64_t m, int64_t n, f32x4_t a, Aux x, Col b) {
    const unsigned d = unsigned(x.y) - unsigned(n);
    const f32x4_t z = a + b;
    if (d < 4) zy[m] = d == 0 ? z[0] : d == 1 ? z[1] : d == 2 ? z[2] : z[3];
    return z;
  }
  __device__ __forceinline__ void operator()(int64_t m, int64_t n, float a) {
    if (int64_t(ylab[m]) == n) zy[m] = bias ? a + bias[n] : a;
  }
  __device__ __forceinline__ void row_stats(int64_t m, int64_t t, float mx, float sum) {
    part[m * tiles + t] = float2{mx, sum};
  }
};

// The same for few rows: z of 64 vocabulary rows and up to 16 · NB hidden rows per workgroup,
// without staging; bound by reading the weight (16 rows, [128256, 4096]: 185 us, 5.7 TB/s). The
// four wavefronts split the columns; each takes v_mfma_f32_16x16x32_bf16 with the weight rows as
// its first operand, so a lane's accumulator is one hidden row's column. A lane loads 32
// consecutive bytes of a weight row per 64 columns (four lanes a full 128-byte line) and the two
// operands share whatever order of k that is. Rows past v and past n repeat the last one; columns
// past h are zero in both operands.
constexpr int kScoreCols = 64;  // vocabulary rows per workgroup
template <int NB>
__global__ void __launch_bounds__(256) score_kernel(
    const uint16_t* __restrict__ hidden, const uint16_t* __restrict__ w,
    const float* __restrict__ bias, const int32_t* __restrict__ labels, int64_t n, int64_t h,
    int64_t v, int64_t v_start, float2* __restrict__ part, int64_t tiles,
    float* __restrict__ zy) {
  constexpr int T = 16 * NB, RB = kScoreCols / 16;
  __shared__ float z[4][kScoreCols][T + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r0 = int64_t(blockIdx.x) * kScoreCols;
  const int64_t span = up((h + 3) / 4, 64);  // columns of one wavefront
  const int64_t k_lo = wave * span + 16 * (lane >> 4);
  const int64_t k_hi = (wave + 1) * span < h ? (wave + 1) * span : h;
  const uint16_t* wp[RB];
  const uint16_t* hp[NB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int64_t r = r0 + 16 * i + (lane & 15);
    wp[i] = w + (r < v ? r : v - 1) * h;
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int64_t r = 16 * j + (lane & 15);
    hp[j] = hidden + (r < n ? r : n - 1) * h;
  }
  f32x4_t acc[RB][NB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto load = [&](const uint16_t* p, int64_t k) {
    const uint4 x = k < h ? *reinterpret_cast<const uint4*>(p + k) : uint4{0u, 0u, 0u, 0u};
    return __builtin_bit_cast(gemm::bf16x8_t, x);
  };
  for (int64_t k0 = wave * span; k0 < k_hi; k0 += 64) {
    const int64_t k = k_lo + (k0 - wave * span);
    gemm::bf16x8_t a[RB][2], b[NB][2];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      a[i][0] = load(wp[i], k);
      a[i][1] = load(wp[i], k + 8);
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      b[j][0] = load(hp[j], k);
      b[j][1] = load(hp[j], k + 8);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i][u], b[j][u], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        z[wave][16 * i + 4 * (lane >> 4) + q][16 * j + (lane & 15)] = acc[i][j][q];
  __syncthreads();
  // 256 / T neighbouring threads share a hidden row, T / 4 vocabulary rows each
  constexpr int kShare = 256 / T, kEach = kScoreCols / kShare;
  const int t = threadIdx.x / kShare, sub = threadIdx.x % kShare;
  const int32_t y = t < n ? labels[t] : -1;
  float x[kEach];
  float m = -INFINITY, s = 0.f;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int c = e * kShare + sub;
    const int64_t r = r0 + c;
    x[e] = ((z[0][c][t] + z[1][c][t]) + z[2][c][t]) + z[3][c][t];
    if (r < v && bias) x[e] += bias[r];
    if (r < v && t < n && int64_t(y) == v_start + r) zy[t] = x[e];
    if (r < v) m = fmaxf(m, x[e]);
  }
  m = fmaxf(m, kLeastMax);
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (r0 + e * kShare + sub < v) s += fast_exp2((x[e] - m) * kLog2e);
#pragma unroll
  for (int off = kShare / 2; off >= 1; off >>= 1) {
    const float m2 = __shfl_xor(m, off, 64), s2 = __shfl_xor(s, off, 64);
    lse_merge(m, s, m2, s2);
  }
  if (sub == 0 && t < n) part[t * tiles + blockIdx.x] = float2{m, s};
}

// One workgroup per row: its tiles' (max, Σ exp) pairs merged in a fixed order, and into the
// state of the pieces before (unless this is the first). `row` maps the rows of `part` to rows
// of the state (NULL: the same, rows without a label set to (−inf, 0, 0)).
__global__ void __launch_bounds__(256) merge_state_kernel(
    const float2* __restrict__ part, int64_t tiles, const float* __restrict__ zy,
    const int32_t* __restrict__ row, const int32_t* __restrict__ count,
    const int32_t* __restrict__ ylab, const int32_t* __restrict__ labels, int64_t n, int64_t v,
    int64_t v_start, int64_t vocab, int32_t ignore_index, int first, float* __restrict__ state) {
  const int64_t m = blockIdx.x;
  int64_t i = m;
  bool here;
  if (row) {
    if (m >= *count) return;
    i = row[m];
    here = ylab[m] >= 0;
  } else {
    const int32_t y = labels[m];
    if (!labelled(y, vocab, ignore_index)) {
      if (first && threadIdx.x == 0) {
        state[i] = -INFINITY;
        state[n + i] = 0.f;
        state[2 * n + i] = 0.f;
      }
      return;
    }
    here = int64_t(y) >= v_start && int64_t(y) < v_start + v;
  }
  float mx = -INFINITY, sum = 0.f;
  for (int64_t t = threadIdx.x; t < tiles; t += 256) {
    const float2 p = part[m * tiles + t];
    lse_merge(mx, sum, p.x, p.y);
  }
  wave_lse_reduce(mx, sum);
  __shared__ float sm[4], ss[4];
  if ((threadIdx.x & 63) == 0) {
    sm[threadIdx.x >> 6] = mx;
    ss[threadIdx.x >> 6] = sum;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  mx = sm[0];
  sum = ss[0];
  for (int w = 1; w < 4; ++w) lse_merge(mx, sum, sm[w], ss[w]);
  float z = here ? zy[m] : 0.f;
  if (!first) {
    float m0 = state[i], s0 = state[n + i];
    lse_merge(m0, s0, mx, sum);
    mx = m0;
    sum = s0;
    if (!here) z = state[2 * n + i];
  }
  state[i] = mx;
  state[n + i] = sum;
  state[2 * n + i] = z;
}

// ------------------------------------------------------------------ loss from the state

struct LossArgs {
  const float* state;
  const int32_t* labels;
  int64_t n, vocab;
  int32_t ignore_index;
  float *lse_out, *row_out;  // NULL: not asked for
};
// Row i's loss term lse − z_y (0 without a label); lse_out and row_out on the way.
__device__ __forceinline__ float loss_term(const LossArgs& a, int64_t i) {
  const int32_t y = a.labels[i];
  float lse = 0.f, term = 0.f;
  if (labelled(y, a.vocab, a.ignore_index)) {
    lse = a.state[i] + fast_log2(a.state[a.n + i]) * kLn2;
    term = lse - a.state[2 * a.n + i];
  }
  if (a.lse_out) a.lse_out[i] = lse;
  if (a.row_out) a.row_out[i] = term;
  return term;
}

// Everything in one workgroup, for few rows: terms, their fp64 sum in a fixed order, the count.
constexpr int kSmallLoss = 4096;
__global__ void __launch_bounds__(1024) small_loss_kernel(LossArgs a, long long t_host,
                                                          float* __restrict__ loss,
                                                          int32_t* __restrict__ status) {
  __shared__ double part[16];
  __shared__ int counts[16];
  __shared__ int any_bad;
  if (threadIdx.x == 0) any_bad = 0;
  __syncthreads();
  double sum = 0.0;
  int count = 0;
  for (int64_t i = threadIdx.x; i < a.n; i += 1024) {
    const int32_t y = a.labels[i];
    if (labelled(y, a.vocab, a.ignore_index))
      ++count;
    else if (y != a.ignore_index)
      any_bad = 1;  // every writer writes the same value
    sum += double(loss_term(a, i));
  }
  sum = wave_sum_f64(sum);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) count += __shfl_xor(count, off, 64);
  if ((threadIdx.x & 63) == 0) {
    part[threadIdx.x >> 6] = sum;
    counts[threadIdx.x >> 6] = count;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  double total = 0.0;
  long long c = 0;
  for (int w = 0; w < 16; ++w) {
    total += part[w];
    c += counts[w];
  }
  const long long t = t_host >= 0 ? t_host : c;
  if (loss) *loss = t > 0 ? float(total / double(t)) : 0.f;
  if (status) *status = any_bad ? LCE_STATUS_BAD_LABEL : 0;
}

__global__ void __launch_bounds__(256) loss_terms_kernel(LossArgs a, float* __restrict__ terms) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.n) return;
  const float t = loss_term(a, i);
  terms[i] = t;
}

// ------------------------------------------------------------------ backward

// D = c · (exp(z − lse) − [v = y]) in bf16, in panels of 64 columns ([np][64] each, so that both
// products read whole 128-byte lines one after the other); 0 in the columns v .. up(v, 64) − 1
// and in the padding rows. What the rounding takes from a label's element goes to left[m]. BIAS: each
// tile's column sums of the fp32 values. ROWS: c is the row's own coefficient, else 1.
template <bool BIAS, bool ROWS>
struct EpiPieceGrad {
  static constexpr bool kRowStats = false, kColSums = BIAS, kTileMax = false, kRowTag = true;
  static constexpr bool kRowLimit = true, kColAux = true;
  uint16_t* d;
  int64_t np;
  const float* bias;
  int64_t v;
  const int32_t* ylab;
  const int32_t* count;
  const float* lse;
  const float* coef;
  float* left;
  float* colsum;
  int64_t v64;
  using Col = f32x4_t;
  struct Aux {
    float lse, c;
    int y;
  };
  __device__ void begin(int64_t) {}
  __device__ __forceinline__ int64_t row_limit() const { return *count; }
  __device__ __forceinline__ int row_tag(int64_t m) const { return ylab[m]; }
  // past the last class: a bias that makes the exponential 0
  __device__ __forceinline__ Col load_col(int64_t n) const {
    Col b = bias4(bias, n, v);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q >= v) b[q] = -INFINITY;
    return b;
  }
  __device__ __forceinline__ Aux load4t(int64_t m, int64_t, int y) const {
    return {lse[m], ROWS ? coef[m] : 1.f, y};
  }
  __device__ __forceinline__ f32x4_t store4c(int64_t m, int64_t n, f32x4_t a, const Aux& x, Col b) {
    const unsigned at = unsigned(x.y) - unsigned(n);
    f32x4_t r;
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = fast_exp2(((a[q] + b[q]) - x.lse) * kLog2e);
    if (at < 4) {  // once a row
      float e = (at == 0 ? r[0] : at == 1 ? r[1] : at == 2 ? r[2] : r[3]) - 1.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = at == unsigned(q) ? e : r[q];
      if (ROWS) e *= x.c;
      left[m] = e - bf16_to_f32(f32_to_bf16(e));
    }
    if (ROWS) {
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] *= x.c;
    }
    *reinterpret_cast<uint2*>(d + (n >> 6) * np * 64 + m * 64 + (n & 63)) =
        uint2{pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3])};
    return r;
  }
  __device__ __forceinline__ void operator()(int64_t, int64_t, float) {}  // N % 4 == 0: unused
  __device__ __forceinline__ void col_sums(int64_t mt, int64_t n, float sum) {
    colsum[mt * v64 + n] = sum;
  }
};

// Where the rows of dH go. The product's row m is the batch's row row[m].
struct HiddenOut {
  const int32_t* row;
  const int32_t* count;
  float* acc;       // fp32 [n, h] over the pieces; NULL with a single piece
  uint16_t* grad;   // bf16 [n, h], written with the last piece (NULL: not)
  int64_t h;
  int first;
  const float* scale;
  const int32_t* ylab;
  const float* left;        // of the labels in this piece: what D's label element lacks
  const uint16_t* weight;   // the piece's rows, ldw apart
  int64_t ldw;
  __device__ __forceinline__ f32x4_t old(int64_t i, int64_t n) const {
    if (first) return f32x4_t{0.f, 0.f, 0.f, 0.f};
    return *reinterpret_cast<const f32x4_t*>(acc + i * h + n);
  }
  __device__ __forceinline__ f32x4_t label(int64_t m, int64_t n) const {
    const int32_t y = ylab[m];
    if (y < 0) return f32x4_t{0.f, 0.f, 0.f, 0.f};
    const uint2 w = *reinterpret_cast<const uint2*>(weight + int64_t(y) * ldw + n);
    return left[m] * f32x4_t{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
  }
  __device__ __forceinline__ void put(int64_t i, int64_t n, f32x4_t x) const {
    if (grad)
      *reinterpret_cast<uint2*>(grad + i * h + n) =
          uint2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    else
      *reinterpret_cast<f32x4_t*>(acc + i * h + n) = x;
  }
};

struct EpiPieceHidden {
  static constexpr bool kRowStats = false, kColSums = false, kTileMax = false, kRowTag = true;
  static constexpr bool kRowLimit = true;
  HiddenOut o;
  float s;
  struct Aux {
    f32x4_t old;
    int i;
  };
  __device__ void begin(int64_t) { s = *o.scale; }
  __device__ __forceinline__ int64_t row_limit() const { return *o.count; }
  __device__ __forceinline__ int row_tag(int64_t m) const {
    return m < int64_t(*o.count) ? o.row[m] : -1;
  }
  __device__ __forceinline__ Aux load4t(int64_t m, int64_t n, int i) const {
    return {i >= 0 ? o.old(i, n) + s * o.label(m, n) : f32x4_t{0.f, 0.f, 0.f, 0.f}, i};
  }
  __device__ __forceinline__ void store4(int64_t, int64_t n, f32x4_t a, const Aux& x) {
    if (x.i >= 0) o.put(x.i, n, x.old + s * a);
  }
  __device__ __forceinline__ void operator()(int64_t, int64_t, float) {}  // h % 4 == 0: unused
};

// The product split over K: partial sums [splits][rows of the tiles that count][h], then added in
// split order. Where fewer rows carry a label than the launch has tiles for, K is cut into as many
// more ranges, of at least kSplitK classes each (a step of 100 rows of 256 and 2000 classes takes
// 112 us with ranges of 1024, 82 with 256): the same workgroups and the same memory.
constexpr int64_t kSplitK = 256;
__host__ __device__ inline int64_t piece_splits(int64_t m_tiles, int64_t live, int64_t splits,
                                                int64_t v) {
  const int64_t most = v / kSplitK > splits ? v / kSplitK : splits;
  const int64_t s = splits * m_tiles / live;
  return s < most ? s : most;
}
struct EpiPiecePartial {
  static constexpr bool kRowStats = false, kColSums = false, kTileMax = false;
  static constexpr bool kRowLimit = true, kResplit = true;
  float* part;
  int64_t h, v;
  const int32_t* count;
  int64_t kz, rows;
  struct Aux {};
  __device__ void begin(int64_t z) {
    kz = z;
    rows = up(*count, kTile);
  }
  __device__ __forceinline__ int64_t row_limit() const { return *count; }
  __device__ __forceinline__ int64_t splits(int64_t m_tiles, int64_t live, int64_t s) const {
    return piece_splits(m_tiles, live, s, v);
  }
  __device__ __forceinline__ Aux load4(int64_t, int64_t) const { return Aux{}; }
  __device__ __forceinline__ void store4(int64_t m, int64_t n, f32x4_t a, Aux) {
    *reinterpret_cast<f32x4_t*>(part + (kz * rows + m) * h + n) = a;
  }
  __device__ __forceinline__ void operator()(int64_t, int64_t, float) {}
};
__device__ __forceinline__ void hidden_reduce(const float* __restrict__ part, int64_t m_tiles,
                                              int64_t splits, int64_t v, const HiddenOut& o,
                                              int64_t block) {
  const int64_t e = (block * 256 + threadIdx.x) * 4;
  const int64_t m = e / o.h, n = e % o.h;
  const int64_t count = *o.count;
  if (m >= count) return;
  const int64_t live = (count + kTile - 1) / kTile;
  splits = piece_splits(m_tiles, live, splits, v);
  f32x4_t a{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int64_t z = 0; z < splits; ++z)
    a += *reinterpret_cast<const f32x4_t*>(part + (z * live * kTile + m) * o.h + n);
  const int64_t i = o.row[m];
  o.put(i, n, o.old(i, n) + *o.scale * (a + o.label(m, n)));
}

// dW (=|+=) s · acc, in bf16 or fp32; the contraction runs over the labelled rows. Where dW is
// overwritten, the rows of the classes that are some row's label (named) hold Σ e_i · hidden_i, what
// D's label elements lack, and the sums start from that.
template <class TW, bool ACC>
struct EpiPieceWeight {
  static constexpr bool kRowStats = false, kColSums = false, kTileMax = false;
  static constexpr bool kKLimit = true, kAccInit = !ACC;
  TW* dw;
  int64_t h;
  const int32_t* count;
  const uint32_t* named;  // a bit a class
  const float* scale;
  float s;
  using Init = std::conditional_t<sizeof(TW) == 4, f32x4_t, u32x2_t>;
  __device__ __forceinline__ uint32_t init_rows(int64_t m) const {
    // uniform, and read only in this launch: by the scalar unit, whose loads wait for no others
    const auto* p = (const __attribute__((address_space(4))) uint32_t*)(named);
    return p[m >> 5] >> (m & 31) & 0xffff;
  }
  __device__ __forceinline__ Init init_load(int64_t m, int64_t n) const {
    return *reinterpret_cast<const Init*>(dw + m * h + n);
  }
  static __device__ __forceinline__ f32x4_t init_value(Init x) {
    if constexpr (sizeof(TW) == 4)
      return x;
    else
      return f32x4_t{bf16_lo(x[0]), bf16_hi(x[0]), bf16_lo(x[1]), bf16_hi(x[1])};
  }
  using Aux = f32x4_t;
  __device__ void begin(int64_t) { s = *scale; }
  __device__ __forceinline__ int64_t k_limit() const { return *count; }
  __device__ __forceinline__ Aux load4(int64_t m, int64_t n) const {
    if constexpr (!ACC) {
      return Aux{0.f, 0.f, 0.f, 0.f};
    } else if constexpr (sizeof(TW) == 4) {
      return *reinterpret_cast<const f32x4_t*>(dw + m * h + n);
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(dw + m * h + n);
      return Aux{bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y)};
    }
  }
  __device__ __forceinline__ void store4(int64_t m, int64_t n, f32x4_t a, Aux old) {
    const f32x4_t x = ACC ? old + s * a : s * a;
    if constexpr (sizeof(TW) == 4)
      *reinterpret_cast<f32x4_t*>(dw + m * h + n) = x;
    else
      *reinterpret_cast<uint2*>(dw + m * h + n) =
          uint2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
  }
  __device__ __forceinline__ void operator()(int64_t, int64_t, float) {}  // h % 4 == 0: unused
};

// db (=|+=) s · the column sums of the row tiles, in tile order.
struct BiasOut {
  const float* colsum;
  int64_t v, v64;
  const int32_t* count;
  const float* scale;
  int accumulate, tile;  // tile: rows that each row of colsum adds up
  float* db;
};
__device__ __forceinline__ void bias_reduce(const BiasOut& o, int64_t block) {
  const int64_t c = block * 256 + threadIdx.x;
  if (c >= o.v) return;
  const int64_t tiles = (int64_t(*o.count) + o.tile - 1) / o.tile;
  float sum = 0.f;
#pragma unroll 4
  for (int64_t t = 0; t < tiles; ++t) sum += o.colsum[t * o.v64 + c];
  const float x = *o.scale * sum;
  o.db[c] = o.accumulate ? o.db[c] + x : x;
}

// What is left after the products: the split hidden gradient added up in the first hidden_blocks
// workgroups, the bias gradient in the others.
__global__ void __launch_bounds__(256) piece_finish_kernel(const float* __restrict__ part,
                                                           int64_t m_tiles, int64_t splits,
                                                           int64_t v, HiddenOut h,
                                                           int64_t hidden_blocks, BiasOut b) {
  const int64_t w = blockIdx.x;
  if (w < hidden_blocks)
    hidden_reduce(part, m_tiles, splits, v, h, w);
  else
    bias_reduce(b, w - hidden_blocks);
}

// ------------------------------------------------------------------ workspaces

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Hidden-gradient splits over K for few output tiles: enough to fill the CUs, each at least
// kSplitK vocabulary rows long.
int64_t hidden_splits(int64_t n, int64_t h, int64_t v) {
  const int64_t tiles = (n + kTile - 1) / kTile * ((h + Wide::BN - 1) / Wide::BN);
  return std::max<int64_t>(1, std::min<int64_t>(256 / std::max<int64_t>(tiles, 1), v / kSplitK));
}

struct PieceWs {
  int32_t *count, *cidx, *row, *ylab;
  uint32_t* named;
  void* order;
  float *zy, *lse_c, *coef_c, *left, *scale, *colsum, *split;
  float2* part;
  uint16_t *hc, *wpad, *d;
  size_t bytes;
};

struct Carver {
  char* base;
  size_t off = 0;
  template <class T>
  T* take(int64_t count) {
    T* p = reinterpret_cast<T*>(base + off);
    off += align256(size_t(count) * sizeof(T));
    return p;
  }
};

// Words of a bit a class, for whole tiles.
int64_t named_words(int64_t v) { return up(v, kTile) / 32; }

PieceWs carve_fwd(void* base, int64_t n, int64_t h, int64_t v) {
  PieceWs w{};
  Carver c{static_cast<char*>(base)};
  if (n <= kScoreRows) {
    w.zy = c.take<float>(n);
    w.part = c.take<float2>(n * ((v + kScoreCols - 1) / kScoreCols));
  } else {
    const int64_t np = up(n, kTile), h64 = up(h, Wide::BK);
    w.count = c.take<int32_t>(1);
    w.cidx = c.take<int32_t>(n);
    w.row = c.take<int32_t>(np);
    w.ylab = c.take<int32_t>(np);
    w.zy = c.take<float>(np);
    // enough for any piece of fewer classes too, whose smaller tiles may be more
    const int64_t few = kFewTiles / ((n + Small::BM - 1) / Small::BM);
    const int64_t tiles = std::max((v + Wide::BN - 1) / Wide::BN,
                                   std::min((v + Small::BN - 1) / Small::BN, few));
    w.part = c.take<float2>(np * tiles);
    w.hc = c.take<uint16_t>(np * h64);
    if (h64 != h) w.wpad = c.take<uint16_t>(v * h64);
  }
  w.bytes = std::max<size_t>(c.off, 256);
  return w;
}

PieceWs carve_bwd(void* base, int64_t n, int64_t h, int64_t v) {
  PieceWs w{};
  Carver c{static_cast<char*>(base)};
  const int64_t np = up(n, kTile), h64 = up(h, Wide::BK), v64 = up(v, 64);
  w.count = c.take<int32_t>(1);
  w.cidx = c.take<int32_t>(n);
  w.row = c.take<int32_t>(np);
  w.ylab = c.take<int32_t>(np);
  w.lse_c = c.take<float>(np);
  w.coef_c = c.take<float>(np);
  w.left = c.take<float>(np);
  w.scale = c.take<float>(1);
  w.hc = c.take<uint16_t>(np * h64);
  if (h64 != h) w.wpad = c.take<uint16_t>(v * h64);
  w.d = c.take<uint16_t>(np * v64);
  w.named = c.take<uint32_t>(named_words(v));
  w.order = c.take<char>(int64_t(embed_weighted_workspace_bytes(n, h)));
  w.colsum = c.take<float>(np / Small::BM * v64);  // as in the forward: for any smaller piece too
  const int64_t splits = hidden_splits(n, h, v);
  if (splits > 1) w.split = c.take<float>(splits * np * h);
  w.bytes = std::max<size_t>(c.off, 256);
  return w;
}

#define PIECE_TRY(expr)                    \
  do {                                     \
    const hipError_t e_ = (expr);          \
    if (e_ != hipSuccess) return e_;       \
  } while (0)

hipError_t rows_and_gather(const uint16_t* hidden, const int32_t* labels, int64_t n, int64_t h,
                           int64_t v, int64_t v_start, int64_t vocab, int32_t ignore_index,
                           const PieceWs& w, float* state, GatherArgs g, hipStream_t s) {
  g.hidden = hidden;
  g.n = n;
  g.h = h;
  g.h64 = up(h, Wide::BK);
  g.count = w.count;
  g.cidx = w.cidx;
  g.row = w.row;
  g.ylab = w.ylab;
  g.hc = w.hc;
  TimedLaunch t(s, K_PIECE_GATHER);
  if (n <= kFewRows) {
    const int each = few_each(n);
    const int64_t blocks = (n + each - 1) / each + kTile / each;
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(unsigned(blocks)), dim3(256), 0, s, g, labels, v, v_start,
                         vocab, ignore_index, each, state);
    };
    if (g.stok)
      launch(gather_few_rows_kernel<true>);
    else
      launch(gather_few_rows_kernel<false>);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(piece_rows_kernel, dim3(1), dim3(1024), 0, s, labels, n, v, v_start, vocab,
                     ignore_index, w.count, w.cidx, w.row, w.ylab, state, g.scale);
  PIECE_TRY(hipGetLastError());
  hipLaunchKernelGGL(gather_rows_kernel, dim3(unsigned(n + kTile)), dim3(256), 0, s, g);
  return hipGetLastError();
}

hipError_t pad_weight(const uint16_t* weight, int64_t h, int64_t v, uint16_t* out, hipStream_t s) {
  TimedLaunch t(s, K_PIECE_GATHER);
  hipLaunchKernelGGL(pad_rows_kernel, dim3(unsigned(std::min(v, kPadGrid))), dim3(256), 0, s,
                     weight, v, h, up(h, Wide::BK), out);
  return hipGetLastError();
}

template <bool BIAS, bool ROWS>
hipError_t grad_logits(const PieceBwdArgs& a, const PieceWs& w, const View& hv, const View& wv,
                       hipStream_t s) {
  const int64_t np = up(a.n, kTile), v64 = up(a.v, 64), h64 = up(a.h, Wide::BK);
  EpiPieceGrad<BIAS, ROWS> e{w.d, np, a.bias, a.v, w.ylab, w.count, w.lse_c, w.coef_c, w.left,
                             w.colsum, v64};
  TimedLaunch t(s, K_PIECE_GRAD_LOGITS);
  if (few_tiles(a.n, a.v))
    return gemm::v2::launch<Small, true, true>(hv, wv, np, v64, h64, 1, true, e, s);
  if (a.n <= kNarrowRows)  // one row tile either way
    return gemm::v2::launch<Narrow, true, true>(hv, wv, np, v64, h64, 1, true, e, s);
  return gemm::v2::launch<Wide, true, true>(hv, wv, np, v64, h64, 1, true, e, s, false, kBand);
}

template <class TW, bool ACC>
hipError_t grad_weight_product(const PieceBwdArgs& a, const PieceWs& w, const View& dv,
                               const View& hv, hipStream_t s) {
  EpiPieceWeight<TW, ACC> e{static_cast<TW*>(a.grad_weight), a.h, w.count, w.named, w.scale, 0.f};
  TimedLaunch t(s, K_PIECE_GRAD_WEIGHT);
  if (few_tiles(a.v, a.h))
    return gemm::v2::launch<Small, false, false>(dv, hv, a.v, a.h, up(a.n, kTile), 1, false, e, s);
  if (a.n <= kShortK)
    return gemm::v2::launch<Pair, false, false>(dv, hv, a.v, a.h, up(a.n, kTile), 1, false, e, s);
  return gemm::v2::launch<Wide, false, false>(dv, hv, a.v, a.h, up(a.n, kTile), 1, true, e, s,
                                              true);
}

// The hidden gradient's product, split over K, and the weight gradient's in one launch: neither
// fills its last round of CUs (steps of 100 rows of 256 and 2000 classes 64 us so and 73 apart, 1000
// of 1024 and 50257 523 and 539, 1500 of 4096 and 32000 1354 and 1389).
template <class TW, bool ACC>
hipError_t grad_products(const PieceBwdArgs& a, const PieceWs& w, const View& dv, const View& wk,
                         const View& hk, int64_t splits, hipStream_t s) {
  const EpiPiecePartial eh{w.split, a.h, a.v, w.count, 0, 0};
  const EpiPieceWeight<TW, ACC> ew{static_cast<TW*>(a.grad_weight), a.h, w.count, w.named, w.scale,
                                   0.f};
  const int64_t np = up(a.n, kTile);
  TimedLaunch t(s, K_PIECE_GRADS);
  return gemm::v2::launch_two<Wide>(
      gemm::v2::product<Wide, true, false>(dv, wk, np, a.h, a.v, splits, true, eh),
      gemm::v2::product<Wide, false, false>(dv, hk, a.v, a.h, np, 1, false, ew), s);
}

}  // namespace

size_t piece_fwd_workspace_bytes(int64_t n, int64_t h, int64_t v) {
  return carve_fwd(nullptr, n, h, v).bytes;
}
size_t piece_bwd_workspace_bytes(int64_t n, int64_t h, int64_t v) {
  return carve_bwd(nullptr, n, h, v).bytes;
}
size_t piece_loss_workspace_bytes(int64_t n) { return ce_workspace_bytes(n); }

hipError_t piece_fwd_run(const PieceFwdArgs& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  const PieceWs w = carve_fwd(a.workspace, a.n, a.h, a.v);
  const int first = (a.flags & FLCE_PIECE_FIRST) != 0;
  int64_t tiles;
  if (a.n <= kScoreRows) {
    tiles = (a.v + kScoreCols - 1) / kScoreCols;
    TimedLaunch t(s, K_PIECE_LOGITS);
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(unsigned(tiles)), dim3(256), 0, s, a.hidden, a.weight,
                         a.bias, a.labels, a.n, a.h, a.v, a.v_start, w.part, tiles, w.zy);
    };
    if (a.n <= 16)
      launch(score_kernel<1>);
    else
      launch(score_kernel<2>);
    PIECE_TRY(hipGetLastError());
  } else {
    tiles = (a.v + lse_cols(a.n, a.v) - 1) / lse_cols(a.n, a.v);
    const int64_t np = up(a.n, kTile), h64 = up(a.h, Wide::BK);
    PIECE_TRY(rows_and_gather(a.hidden, a.labels, a.n, a.h, a.v, a.v_start, a.vocab,
                              a.ignore_index, w, first ? a.state : nullptr, GatherArgs{}, s));
    const uint16_t* weight = a.weight;
    if (w.wpad) {
      PIECE_TRY(pad_weight(a.weight, a.h, a.v, w.wpad, s));
      weight = w.wpad;
    }
    View hv{w.hc, h64, 64, np, h64};
    View wv{weight, h64, 64, a.v, h64};
    EpiPieceLse e{a.bias, a.v, w.ylab, w.count, w.part, tiles, w.zy};
    TimedLaunch t(s, K_PIECE_LOGITS);
    if (few_tiles(a.n, a.v))
      PIECE_TRY((gemm::v2::launch<Small, true, true>(hv, wv, np, a.v, h64, 1, true, e, s)));
    else if (a.n <= kNarrowRows)
      PIECE_TRY((gemm::v2::launch<Narrow, true, true>(hv, wv, np, a.v, h64, 1, true, e, s)));
    else
      PIECE_TRY((gemm::v2::launch<Wide, true, true>(hv, wv, np, a.v, h64, 1, true, e, s, false,
                                                    kBand)));
  }
  TimedLaunch t(s, K_PIECE_STATE);
  hipLaunchKernelGGL(merge_state_kernel, dim3(unsigned(a.n)), dim3(256), 0, s, w.part, tiles, w.zy,
                     w.row, w.count, w.ylab, a.labels, a.n, a.v, a.v_start, a.vocab,
                     a.ignore_index, first, a.state);
  return hipGetLastError();
}

hipError_t piece_loss_run(const PieceLossArgs& a, hipStream_t s) {
  const LossArgs l{a.state, a.labels, a.n, a.vocab, a.ignore_index, a.lse_out, a.row_loss_out};
  const long long th = a.num_label_tokens >= 0 ? a.num_label_tokens : -1;
  if (a.n <= kSmallLoss) {
    TimedLaunch t(s, K_PIECE_STATE);
    hipLaunchKernelGGL(small_loss_kernel, dim3(1), dim3(1024), 0, s, l, th, a.loss_out,
                       a.status_out);
    return hipGetLastError();
  }
  const CeWorkspace ws = ce_workspace_carve(a.workspace, a.n);
  PIECE_TRY(launch_label_prep(a.labels, a.n, a.vocab, a.ignore_index, ws.count, a.status_out, s));
  {
    TimedLaunch t(s, K_PIECE_STATE);
    hipLaunchKernelGGL(loss_terms_kernel, dim3(unsigned((a.n + 255) / 256)), dim3(256), 0, s, l,
                       ws.row_loss);
    PIECE_TRY(hipGetLastError());
  }
  if (!a.loss_out) return hipSuccess;
  return launch_loss_reduce(ws.row_loss, a.n, ws.count, th, a.loss_out, s);
}

hipError_t piece_bwd_run(const PieceBwdArgs& a, hipStream_t s) {
  const bool first = (a.flags & FLCE_PIECE_FIRST) != 0, last = (a.flags & FLCE_PIECE_LAST) != 0;
  const bool accumulate = (a.flags & FLCE_PIECE_ACCUMULATE) != 0;
  const PieceWs w = carve_bwd(a.workspace, a.n, a.h, a.v);
  const int64_t np = up(a.n, kTile), h64 = up(a.h, Wide::BK), v64 = up(a.v, 64);
  const bool rows = a.grad_rows != nullptr;
  const bool want_weight = a.grad_weight && !(a.n == 0 && accumulate);
  const bool wide = a.grad_weight_dtype == LCE_DTYPE_F32;
  // what the labels' elements lack goes into the weight gradient too, but a bf16 one that is added
  // to has no bits for it
  const bool want_labels = want_weight && (wide || !accumulate);
  GatherArgs g{};
  g.words = named_words(a.v);
  if (want_labels) {
    g.named = accumulate ? nullptr : w.named;
    if (a.n <= kFewRows) embed_weighted_order(w.order, a.n, a.h, &g.stok, &g.spos);
  }
  g.lse = a.lse;
  g.grad_rows = a.grad_rows;
  g.lse_c = w.lse_c;
  g.coef_c = rows ? w.coef_c : nullptr;
  g.row_scale = w.scale;
  g.scale = ScaleOut{rows ? nullptr : w.scale, a.num_label_tokens, a.grad_output};
  uint16_t* const grad_hidden = last ? a.grad_hidden : nullptr;
  g.zero_acc = first && !grad_hidden ? a.hidden_acc : nullptr;
  g.zero_grad = grad_hidden;
  if (rows) {
    TimedLaunch t(s, K_PIECE_GATHER);
    hipLaunchKernelGGL(row_scale_kernel, dim3(1), dim3(1024), 0, s, a.grad_rows, a.labels, a.n,
                       a.vocab, a.ignore_index, w.scale);
    PIECE_TRY(hipGetLastError());
  }
  PIECE_TRY(rows_and_gather(a.hidden, a.labels, a.n, a.h, a.v, a.v_start, a.vocab, a.ignore_index,
                            w, nullptr, g, s));
  const uint16_t* weight = a.weight;
  if (w.wpad) {
    PIECE_TRY(pad_weight(a.weight, a.h, a.v, w.wpad, s));
    weight = w.wpad;
  }
  View hv{w.hc, h64, 64, np, h64};
  View wv{weight, h64, 64, a.v, h64};
  if (a.n > 0) {
    if (a.grad_bias)
      PIECE_TRY((rows ? grad_logits<true, true>(a, w, hv, wv, s)
                      : grad_logits<true, false>(a, w, hv, wv, s)));
    else
      PIECE_TRY((rows ? grad_logits<false, true>(a, w, hv, wv, s)
                      : grad_logits<false, false>(a, w, hv, wv, s)));
  }
  View dv{w.d, 64, np * 64, np, a.v};
  dv.ext = np * v64;
  View wk{weight, h64, 64, a.v, a.h};
  View hk{w.hc, h64, 64, np, a.h};
  const bool want_hidden = a.n > 0 && (grad_hidden || a.hidden_acc);
  const int64_t splits = hidden_splits(a.n, a.h, a.v);
  if (want_labels && a.n > 0) {
    const EmbedBwdArgs e{w.hc, LCE_DTYPE_BF16, h64, w.ylab, a.n, a.h, a.v, -1, 1.f,
                         accumulate ? EMBED_ACCUMULATE : 0, a.grad_weight, a.grad_weight_dtype,
                         a.h, nullptr, w.order};
    // overwritten, dW takes s with the product
    PIECE_TRY(embed_weighted_run(e, w.left, accumulate ? w.scale : nullptr, g.stok != nullptr,
                                 accumulate ? nullptr : w.named, s));
  }
  const bool both = want_hidden && want_weight && splits > 1 && !few_tiles(a.v, a.h);
  const HiddenOut o{w.row, w.count, a.hidden_acc, grad_hidden, a.h,
                    int(first), w.scale, w.ylab, w.left, weight, h64};
  if (both) {
    if (wide)
      PIECE_TRY((accumulate ? grad_products<float, true>(a, w, dv, wk, hk, splits, s)
                            : grad_products<float, false>(a, w, dv, wk, hk, splits, s)));
    else
      PIECE_TRY((accumulate ? grad_products<uint16_t, true>(a, w, dv, wk, hk, splits, s)
                            : grad_products<uint16_t, false>(a, w, dv, wk, hk, splits, s)));
  } else if (want_hidden) {
    TimedLaunch t(s, K_PIECE_GRAD_HIDDEN);
    if (splits == 1) {
      EpiPieceHidden e{o, 0.f};
      PIECE_TRY((gemm::v2::launch<Wide, true, false>(dv, wk, np, a.h, a.v, 1, true, e, s, true)));
    } else {
      EpiPiecePartial e{w.split, a.h, a.v, w.count, 0, 0};
      PIECE_TRY((gemm::v2::launch<Wide, true, false>(dv, wk, np, a.h, a.v, splits, true, e, s)));
    }
  }
  if (want_weight && !both) {
    if (wide)
      PIECE_TRY((accumulate ? grad_weight_product<float, true>(a, w, dv, hk, s)
                            : grad_weight_product<float, false>(a, w, dv, hk, s)));
    else
      PIECE_TRY((accumulate ? grad_weight_product<uint16_t, true>(a, w, dv, hk, s)
                            : grad_weight_product<uint16_t, false>(a, w, dv, hk, s)));
  }
  const bool want_bias = a.grad_bias && !(a.n == 0 && accumulate);
  const int64_t hidden_blocks = want_hidden && splits > 1 ? (a.n * a.h / 4 + 255) / 256 : 0;
  const int64_t bias_blocks = want_bias ? (a.v + 255) / 256 : 0;
  if (hidden_blocks + bias_blocks > 0) {
    const BiasOut b{w.colsum, a.v, v64, w.count, w.scale, int(accumulate), grad_rows(a.n, a.v),
                    a.grad_bias};
    TimedLaunch t(s, K_PIECE_GRAD_FINISH);
    hipLaunchKernelGGL(piece_finish_kernel, dim3(unsigned(hidden_blocks + bias_blocks)), dim3(256),
                       0, s, w.split, np / kTile, splits, a.v, o, hidden_blocks, b);
    PIECE_TRY(hipGetLastError());
  }
  return hipSuccess;
}

}  // namespace lce
