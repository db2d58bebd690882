// extern "C" entry points of the root-mean-square norm, 8-bit product and beam search operators:
// argument validation, all of it before any HIP call, then the launch code in rms_kernels.hip,
// fp8_kernels.hip and beam_kernels.hip.
#include <algorithm>
#include <limits>
#include <new>
#include <utility>
#include <vector>

#include "capi_checks.h"
#include "common.h"
#include "lce_masked.h"
#include "ops.h"

namespace {

using namespace lce;

constexpr int64_t kI32Max = std::numeric_limits<int32_t>::max();

// Bytes of an element, 0 for an unknown type.
int64_t dtype_size(int dtype) {
  return dtype == LCE_DTYPE_BF16 || dtype == LCE_DTYPE_F16 ? 2 : dtype == LCE_DTYPE_F32 ? 4 : 0;
}
int64_t scale_size(int dtype) {
  return dtype == LCE_SCALE_E8M0 ? 1 : dtype == LCE_SCALE_F32 ? 4 : 0;
}

bool matrix_fits(int64_t rows, int64_t ld) {
  return !mul_overflows(rows, ld) && !mul_overflows(rows * ld, 4);
}

int64_t blocks_of(int64_t h) { return (h + 127) / 128; }

int rms_check_shape(int64_t n, int64_t h) {
  return n < 0 || n > kI32Max || h < 1 || h > LAYERNORM_MAX_H ? LCE_ERR_BAD_SHAPE : LCE_OK;
}

// Whether two row sets are the same ones, or share no bytes.
bool same_or_apart(const void* p, int64_t ldp, Span sp, const void* q, int64_t ldq, Span sq) {
  return (p == q && ldp == ldq) || !spans_meet(sp, sq);
}

int rms_fwd(const void* x, int dtype, int64_t n, int64_t h, int64_t ldx, const void* residual,
            int64_t ldr, const void* weight, int param_dtype, float eps, void* y, int64_t ldy,
            bool fp8, void* scales, int scale_dtype, int64_t lds, void* residual_out,
            int64_t ldro, float* rstd_out, void* stream) {
  int rc = rms_check_shape(n, h);
  if (rc != LCE_OK) return rc;
  const int64_t el = dtype_size(dtype), pl = dtype_size(param_dtype);
  const int64_t sl = fp8 ? scale_size(scale_dtype) : 1, yl = fp8 ? 1 : el;
  if (!el || !pl || !sl || (param_dtype != dtype && param_dtype != LCE_DTYPE_F32))
    return LCE_ERR_BAD_DTYPE;
  if (ldx < h || ldy < h || !matrix_fits(n, ldx) || !matrix_fits(n, ldy) || !(eps >= 0.f) ||
      (residual && (ldr < h || !matrix_fits(n, ldr))) ||
      (residual_out && (ldro < h || !matrix_fits(n, ldro))) ||
      (fp8 && (lds < n || !matrix_fits(blocks_of(h), lds))))
    return LCE_ERR_BAD_SHAPE;
  if (n > 0 && (!x || !y || (fp8 && !scales))) return LCE_ERR_NULL_ARG;
  if (!aligned(x, el) || !aligned(residual, el) || !aligned(weight, pl) || !aligned(y, yl) ||
      !aligned(residual_out, el) || !aligned(rstd_out, 4) || (fp8 && !aligned(scales, sl)))
    return LCE_ERR_ALIGNMENT;
  {
    const Span sx = span(x, matrix_bytes(n, ldx, h, el));
    const Span sr = span(residual, residual ? matrix_bytes(n, ldr, h, el) : 0);
    const Span sy = span(y, matrix_bytes(n, ldy, h, yl));
    const Span so = span(residual_out, residual_out ? matrix_bytes(n, ldro, h, el) : 0);
    const Span wr[] = {sy, so, span(rstd_out, 4 * n),
                       span(fp8 ? scales : nullptr,
                            fp8 ? matrix_bytes(blocks_of(h), lds, n, sl) : 0)};
    const Span rd[] = {span(weight, pl * h)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
    for (const Span& w : {wr[2], wr[3]})
      if (spans_meet(w, sx) || spans_meet(w, sr)) return LCE_ERR_OVERLAP;
    if (!same_or_apart(residual_out, ldro, so, x, ldx, sx) ||
        !same_or_apart(residual_out, ldro, so, residual, ldr, sr))
      return LCE_ERR_OVERLAP;
    if (fp8 ? spans_meet(sy, sx) || spans_meet(sy, sr)
            : !same_or_apart(y, ldy, sy, x, ldx, sx) ||
                  !same_or_apart(y, ldy, sy, residual, ldr, sr))
      return LCE_ERR_OVERLAP;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const RmsFwdArgs a{x, dtype, n, h, ldx, residual, ldr, weight, param_dtype, eps, y, ldy,
                     residual_out, ldro, rstd_out, fp8 ? scales : nullptr, scale_dtype, lds};
  LCE_TRY_HIP(rmsnorm_fwd_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int matmul_check_shape(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || m > (int64_t(1) << 23) || n < 1 || n > (int64_t(1) << 28) || k < 16 ||
      k % 16 != 0 || k > (int64_t(1) << 20) ||
      (m + 255) / 256 * ((n + 255) / 256) >= (int64_t(1) << 22))  // small tiles: 2^32 threads
    return LCE_ERR_BAD_SHAPE;
  return LCE_OK;
}

int matmul(const uint8_t* a, int64_t lda, const void* a_scales, int64_t ldas, const uint8_t* b,
           int64_t ldb, const void* b_scales, int64_t ldbs, int scale_dtype, const float* bias,
           int64_t m, int64_t n, int64_t k, void* out, int out_dtype, int64_t ldo, void* workspace,
           size_t workspace_bytes, bool precise, void* stream) {
  int rc = matmul_check_shape(m, n, k);
  if (rc != LCE_OK) return rc;
  const int64_t sl = scale_size(scale_dtype), ol = dtype_size(out_dtype);
  if (!sl || !ol) return LCE_ERR_BAD_DTYPE;
  const int64_t blocks = blocks_of(k), widest = int64_t(1) << 22;
  if (lda < k || lda > widest || lda % 16 != 0 || ldb < k || ldb > widest || ldb % 16 != 0 ||
      ldo < n || ldas < m || ldbs < blocks || !matrix_fits(m, ldo) || !matrix_fits(blocks, ldas) ||
      !matrix_fits(blocks_of(n), ldbs) || ldbs > widest)
    return LCE_ERR_BAD_SHAPE;
  if (!b || !b_scales || (m > 0 && (!a || !a_scales || !out))) return LCE_ERR_NULL_ARG;
  const size_t need = fp8_matmul_workspace_bytes(m, n, k);
  if (need > 0 && (!workspace || workspace_bytes < need)) return LCE_ERR_WORKSPACE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scales, sl) || !aligned(b_scales, sl) ||
      !aligned(bias, 4) || !aligned(out, ol) || (need > 0 && !aligned(workspace, 256)))
    return LCE_ERR_ALIGNMENT;
  {
    const Span wr[] = {span(need > 0 ? workspace : nullptr, int64_t(need)),
                       span(out, matrix_bytes(m, ldo, n, ol))};
    const Span rd[] = {span(a, matrix_bytes(m, lda, k, 1)), span(b, matrix_bytes(n, ldb, k, 1)),
                       span(a_scales, m > 0 ? matrix_bytes(blocks, ldas, m, sl) : 0),
                       span(b_scales, matrix_bytes(blocks_of(n), ldbs, blocks, sl)),
                       span(bias, 4 * n)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const Fp8MatmulArgs args{a,    lda, a_scales, ldas, b,   ldb,       b_scales, ldbs,      scale_dtype,
                           bias, m,   n,        k,    out, out_dtype, ldo,      workspace, precise};
  LCE_TRY_HIP(fp8_matmul_run(args, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int beam_check_shape(int64_t batch, int64_t beams, int64_t v, int64_t num) {
  if (batch < 0 || batch > kI32Max || beams < 1 || beams > BEAM_MAX_BEAMS || v < 1 ||
      v > kI32Max || num < 1 || num > BEAM_MAX_CANDIDATES)
    return LCE_ERR_BAD_SHAPE;
  return batch > 0 && beam_step_slices(batch * beams, v) >= (int64_t(1) << 23)
             ? LCE_ERR_BAD_SHAPE
             : LCE_OK;
}

// Bytes from the first to the last of a state, -1 where they do not fit.
int64_t state_bytes(int64_t batch, int64_t slots, int64_t entry, int64_t beam, int64_t segment,
                    int64_t segments, int64_t bytes) {
  constexpr int64_t kMost = int64_t(1) << 50;
  const int64_t dims[] = {batch, slots, segments}, strides[] = {entry, beam, segment};
  int64_t total = bytes;
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0 || (strides[i] > 0 && dims[i] - 1 > kMost / strides[i])) return -1;
    total += (dims[i] - 1) * strides[i];
    if (total > kMost) return -1;
  }
  return total;
}

// Whether the runs of a state lie apart from one another: of its three strides in rising order,
// each holds all that the smaller ones span.
bool runs_apart(int64_t batch, int64_t slots, int64_t entry, int64_t beam, int64_t segment,
                int64_t segments, int64_t bytes) {
  int64_t dims[] = {batch, slots, segments}, strides[] = {entry, beam, segment};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (strides[j] > strides[j + 1]) {
        std::swap(strides[j], strides[j + 1]);
        std::swap(dims[j], dims[j + 1]);
      }
  int64_t size = bytes;
  for (int i = 0; i < 3; ++i) {
    if (dims[i] <= 1) continue;
    if (strides[i] < size) return false;
    size += (dims[i] - 1) * strides[i];
  }
  return true;
}

// What a call reads or writes of one state: runs of `bytes` bytes at at.lo plus multiples of the
// strides.
struct Used {
  Span at;  // from the first byte to behind the last
  bool written;
  int64_t bytes;
  int64_t dims[3], strides[3];
};

// Whether two such sets share a byte. A run of one at offset x of its start and one of the other at
// offset y meet where x - y lies in (d - a.bytes, d + b.bytes), d the distance of the starts; x - y
// is a sum of multiples of the strides. They are tried from the longest stride on, as far as the
// shorter ones can make up for it: for strides that hold what the shorter ones span, two or three
// multiples of each. `steps` bounds the work of a call; without any left the answer is yes.
struct Meet {
  int64_t strides[6], least[6], most[6];  // and the multiples of each
  int64_t low[7], high[7];                // what a stride and the shorter ones may add up to
  int terms = 0;
  int64_t* steps;

  void add(int64_t stride, int64_t from, int64_t to) {
    if (stride == 0 || from == to) return;
    int k = 0;
    while (k < terms && strides[k] != stride) ++k;
    if (k == terms) {
      strides[terms] = stride;
      least[terms] = most[terms] = 0;
      ++terms;
    }
    least[k] += from;
    most[k] += to;
  }
  // Whether some sum of the terms from k on lies in [from, to].
  bool some(int k, int64_t from, int64_t to) const {
    if (from > high[k] || to < low[k]) return false;
    if (k == terms) return true;  // the empty sum, 0
    if (--*steps < 0) return true;
    const int64_t s = strides[k];
    // from - high[k + 1] <= t s <= to - low[k + 1]
    const int64_t a = from - high[k + 1], b = to - low[k + 1];
    const int64_t first = std::max(least[k], a >= 0 ? (a + s - 1) / s : -(-a / s));
    const int64_t last = std::min(most[k], b >= 0 ? b / s : -((-b + s - 1) / s));
    for (int64_t t = first; t <= last; ++t)
      if (some(k + 1, from - t * s, to - t * s)) return true;
    return false;
  }
};
bool share_bytes(const Used& a, const Used& b, int64_t* steps) {
  Meet m;
  m.steps = steps;
  for (int i = 0; i < 3; ++i) {
    m.add(a.strides[i], 0, a.dims[i] - 1);
    m.add(b.strides[i], 1 - b.dims[i], 0);
  }
  for (int i = 0; i < m.terms; ++i)
    for (int j = 0; j + 1 < m.terms - i; ++j)
      if (m.strides[j] < m.strides[j + 1]) {
        std::swap(m.strides[j], m.strides[j + 1]);
        std::swap(m.least[j], m.least[j + 1]);
        std::swap(m.most[j], m.most[j + 1]);
      }
  m.low[m.terms] = m.high[m.terms] = 0;
  for (int k = m.terms - 1; k >= 0; --k) {
    m.low[k] = m.low[k + 1] + m.least[k] * m.strides[k];
    m.high[k] = m.high[k + 1] + m.most[k] * m.strides[k];
  }
  const int64_t d = b.at.lo >= a.at.lo ? int64_t(b.at.lo - a.at.lo) : -int64_t(a.at.lo - b.at.lo);
  return m.some(0, d - a.bytes + 1, d + b.bytes - 1);
}

// Whether anything written shares a byte with what is read or with another that is written. In the
// order of their starts a range that meets an earlier one starts before that one's end: where none
// does, that is all. States that interlace (keys and values in one tensor, say) are then looked at
// pair by pair; too many of them for kMeetSteps count as sharing.
// `open`: room for as many indices, those of the ranges that have not ended.
constexpr int64_t kMeetSteps = int64_t(1) << 20;
bool written_meets(std::vector<Used>& all, std::vector<size_t>& open) {
  std::sort(all.begin(), all.end(),
            [](const Used& a, const Used& b) { return a.at.lo < b.at.lo; });
  uintptr_t read_to = 0, written_to = 0;
  int64_t steps = kMeetSteps;
  for (size_t i = 0; i < all.size(); ++i) {
    const Used& u = all[i];
    if (u.at.lo < written_to || (u.written && u.at.lo < read_to)) {
      open.erase(std::remove_if(open.begin(), open.end(),
                                [&](size_t j) { return all[j].at.hi <= u.at.lo; }),
                 open.end());
      for (size_t j : open) {
        if (--steps < 0) return true;
        if ((u.written || all[j].written) && share_bytes(all[j], u, &steps)) return true;
      }
    }
    open.push_back(i);
    uintptr_t& to = u.written ? written_to : read_to;
    to = std::max(to, u.at.hi);
  }
  return false;
}

}  // namespace

extern "C" {

int rmsnorm_fwd(const void* x, int dtype, int64_t n, int64_t h, int64_t ldx, const void* residual,
                int64_t ldr, const void* weight, int param_dtype, float eps, void* y, int64_t ldy,
                void* residual_out, int64_t ldro, float* rstd_out, void* stream) {
  return rms_fwd(x, dtype, n, h, ldx, residual, ldr, weight, param_dtype, eps, y, ldy, false,
                 nullptr, LCE_SCALE_F32, 0, residual_out, ldro, rstd_out, stream);
}

int rmsnorm_fp8_fwd(const void* x, int dtype, int64_t n, int64_t h, int64_t ldx,
                    const void* residual, int64_t ldr, const void* weight, int param_dtype,
                    float eps, uint8_t* q, int64_t ldq, void* scales, int scale_dtype,
                    int64_t lds, void* residual_out, int64_t ldro, float* rstd_out,
                    void* stream) {
  return rms_fwd(x, dtype, n, h, ldx, residual, ldr, weight, param_dtype, eps, q, ldq, true,
                 scales, scale_dtype, lds, residual_out, ldro, rstd_out, stream);
}

int rmsnorm_workspace_size(int64_t n, int64_t h, size_t* bytes) {
  if (!bytes) return LCE_ERR_NULL_ARG;
  const int rc = rms_check_shape(n, h);
  if (rc != LCE_OK) return rc;
  *bytes = rmsnorm_workspace_bytes(n, h);
  return LCE_OK;
}

int rmsnorm_bwd(const void* grad, int dtype, int64_t ldg, const void* x, int64_t ldx,
                const float* rstd, const void* weight, int param_dtype, const void* grad_residual,
                int64_t ldgr, int64_t n, int64_t h, uint32_t flags, void* grad_x, int64_t lddx,
                void* grad_weight, int grad_param_dtype, void* workspace, size_t workspace_bytes,
                void* stream) {
  if (flags & ~RMSNORM_ACCUMULATE) return LCE_ERR_BAD_FLAGS;
  int rc = rms_check_shape(n, h);
  if (rc != LCE_OK) return rc;
  const int64_t el = dtype_size(dtype), pl = dtype_size(param_dtype),
                gl = dtype_size(grad_param_dtype);
  if (!el || !pl || !gl || (param_dtype != dtype && param_dtype != LCE_DTYPE_F32) ||
      (grad_param_dtype != param_dtype && grad_param_dtype != LCE_DTYPE_F32))
    return LCE_ERR_BAD_DTYPE;
  if (ldg < h || ldx < h || !matrix_fits(n, ldg) || !matrix_fits(n, ldx) ||
      (grad_x && (lddx < h || !matrix_fits(n, lddx))) ||
      (grad_residual && (ldgr < h || !matrix_fits(n, ldgr))))
    return LCE_ERR_BAD_SHAPE;
  if (n > 0 && (!grad || !x || !rstd)) return LCE_ERR_NULL_ARG;
  const size_t need = grad_weight ? rmsnorm_workspace_bytes(n, h) : 0;
  if (grad_weight && (!workspace || workspace_bytes < need)) return LCE_ERR_WORKSPACE;
  if (!aligned(grad, el) || !aligned(x, el) || !aligned(grad_x, el) || !aligned(rstd, 4) ||
      !aligned(grad_residual, el) || !aligned(weight, pl) || !aligned(grad_weight, gl) ||
      (grad_weight && !aligned(workspace, 256)))
    return LCE_ERR_ALIGNMENT;
  {
    const Span sg = span(grad, matrix_bytes(n, ldg, h, el));
    const Span ss = span(grad_residual, grad_residual ? matrix_bytes(n, ldgr, h, el) : 0);
    const Span sd = span(grad_x, grad_x ? matrix_bytes(n, lddx, h, el) : 0);
    const Span wr[] = {sd, span(grad_weight ? workspace : nullptr, int64_t(need)),
                       span(grad_weight, gl * h)};
    const Span rd[] = {span(x, matrix_bytes(n, ldx, h, el)), span(rstd, 4 * n),
                       span(weight, pl * h)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
    for (const Span& w : {wr[1], wr[2]})
      if (spans_meet(w, sg) || spans_meet(w, ss)) return LCE_ERR_OVERLAP;
    if (!same_or_apart(grad_x, lddx, sd, grad, ldg, sg) ||
        !same_or_apart(grad_x, lddx, sd, grad_residual, ldgr, ss))
      return LCE_ERR_OVERLAP;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const RmsBwdArgs a{grad, dtype, ldg, x, ldx, rstd, weight, param_dtype, grad_residual, ldgr, n,
                     h, flags, grad_x, lddx, grad_weight, grad_param_dtype, workspace};
  LCE_TRY_HIP(rmsnorm_bwd_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int fp8_quantize(const void* x, int dtype, int64_t n, int64_t h, int64_t ldx, int64_t block_rows,
                 uint8_t* q, int64_t ldq, void* scales, int scale_dtype, int64_t lds,
                 void* stream) {
  if (n < 0 || n > kI32Max || h < 1 || h > (int64_t(1) << 20) || n * h > (int64_t(1) << 34) ||
      (block_rows != 1 && block_rows != 128) ||
      fp8_quantize_groups(n, h, block_rows) >= (int64_t(1) << 24))  // 2^32 threads
    return LCE_ERR_BAD_SHAPE;
  const int64_t el = dtype_size(dtype), sl = scale_size(scale_dtype);
  if (!el || !sl) return LCE_ERR_BAD_DTYPE;
  const int64_t srows = block_rows == 1 ? blocks_of(h) : blocks_of(n);
  const int64_t scols = block_rows == 1 ? n : blocks_of(h);
  if (ldx < h || ldq < h || lds < scols || !matrix_fits(n, ldx) || !matrix_fits(n, ldq) ||
      !matrix_fits(srows, lds))
    return LCE_ERR_BAD_SHAPE;
  if (n > 0 && (!x || !q || !scales)) return LCE_ERR_NULL_ARG;
  if (!aligned(x, el) || !aligned(scales, sl)) return LCE_ERR_ALIGNMENT;
  int rc;
  {
    const Span wr[] = {span(q, matrix_bytes(n, ldq, h, 1)),
                       span(scales, matrix_bytes(srows, lds, scols, sl))};
    const Span rd[] = {span(x, matrix_bytes(n, ldx, h, el))};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const Fp8QuantizeArgs a{x, dtype, n, h, ldx, block_rows, q, ldq, scales, scale_dtype, lds};
  LCE_TRY_HIP(fp8_quantize_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int fp8_matmul_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes) return LCE_ERR_NULL_ARG;
  const int rc = matmul_check_shape(m, n, k);
  if (rc != LCE_OK) return rc;
  *bytes = fp8_matmul_workspace_bytes(m, n, k);
  return LCE_OK;
}

int fp8_matmul(const uint8_t* a, int64_t lda, const void* a_scales, int64_t ldas,
               const uint8_t* b, int64_t ldb, const void* b_scales, int64_t ldbs, int scale_dtype,
               const float* bias, int64_t m, int64_t n, int64_t k, void* out, int out_dtype,
               int64_t ldo, void* workspace, size_t workspace_bytes, void* stream) {
  return matmul(a, lda, a_scales, ldas, b, ldb, b_scales, ldbs, scale_dtype, bias, m, n, k, out,
                out_dtype, ldo, workspace, workspace_bytes, false, stream);
}

int fp8_matmul_precise(const uint8_t* a, int64_t lda, const void* a_scales, int64_t ldas,
                       const uint8_t* b, int64_t ldb, const void* b_scales, int64_t ldbs,
                       int scale_dtype, const float* bias, int64_t m, int64_t n, int64_t k,
                       void* out, int out_dtype, int64_t ldo, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return matmul(a, lda, a_scales, ldas, b, ldb, b_scales, ldbs, scale_dtype, bias, m, n, k, out,
                out_dtype, ldo, workspace, workspace_bytes, true, stream);
}

int beam_step_workspace_size(int64_t batch, int64_t beams, int64_t v, int64_t num, size_t* bytes) {
  if (!bytes) return LCE_ERR_NULL_ARG;
  const int rc = beam_check_shape(batch, beams, v, num);
  if (rc != LCE_OK) return rc;
  *bytes = batch > 0 ? beam_step_workspace_bytes(batch, beams, v, num) : 0;
  return LCE_OK;
}

int beam_step(const void* logits, int dtype, int64_t batch, int64_t beams, int64_t v, int64_t ldl,
              const float* scores, const uint8_t* finished, int32_t eos, int64_t num,
              int32_t ignore_index, float* scores_out, int32_t* parents_out, int32_t* tokens_out,
              uint8_t* finished_out, int32_t* status_out, void* workspace, size_t workspace_bytes,
              void* stream) {
  int rc = beam_check_shape(batch, beams, v, num);
  if (rc != LCE_OK) return rc;
  const int64_t el = dtype_size(dtype), rows = batch * beams;
  if (!el) return LCE_ERR_BAD_DTYPE;
  if (ldl < v || !matrix_fits(rows, ldl) || eos >= v || (finished && eos < 0))
    return LCE_ERR_BAD_SHAPE;
  if (batch > 0 && (!logits || !scores || !scores_out || !parents_out || !tokens_out))
    return LCE_ERR_NULL_ARG;
  const size_t need = batch > 0 ? beam_step_workspace_bytes(batch, beams, v, num) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return LCE_ERR_WORKSPACE;
  if (!aligned(logits, el) || !aligned(scores, 4) || !aligned(scores_out, 4) ||
      !aligned(parents_out, 4) || !aligned(tokens_out, 4) || !aligned(status_out, 4) ||
      (need > 0 && !aligned(workspace, 256)))
    return LCE_ERR_ALIGNMENT;
  {
    const int64_t outs = batch * num;
    const Span wr[] = {span(need > 0 ? workspace : nullptr, int64_t(need)),
                       span(scores_out, 4 * outs), span(parents_out, 4 * outs),
                       span(tokens_out, 4 * outs), span(finished_out, outs), span(status_out, 4)};
    const Span rd[] = {span(logits, matrix_bytes(rows, ldl, v, el)), span(scores, 4 * rows),
                       span(finished, rows)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const BeamStepArgs a{logits, dtype, batch, beams, v, ldl, scores, finished, eos, num,
                       ignore_index, scores_out, parents_out, tokens_out, finished_out,
                       status_out, workspace};
  LCE_TRY_HIP(beam_step_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int beam_reorder(const lce_beam_state* states, int64_t count, const int32_t* parents,
                 int64_t batch, int64_t beams, int64_t slots, void* stream) {
  if (count < 0 || count > (int64_t(1) << 16) || batch < 0 || batch > kI32Max || beams < 1 ||
      beams > BEAM_MAX_BEAMS || slots < 1 || slots > BEAM_MAX_BEAMS)
    return LCE_ERR_BAD_SHAPE;
  if (count > 0 && !states) return LCE_ERR_NULL_ARG;
  if (count == 0 || batch == 0) return LCE_OK;
  if (!parents) return LCE_ERR_NULL_ARG;
  if (!aligned(parents, 4)) return LCE_ERR_ALIGNMENT;
  std::vector<Used> used;
  std::vector<size_t> open;
  try {
    used.reserve(2 * size_t(count) + 1);
    open.reserve(2 * size_t(count) + 1);
  } catch (const std::bad_alloc&) {
    return LCE_ERR_SCRATCH_LIMIT;
  }
  used.push_back({span(parents, 4 * batch * slots), false, 4 * batch * slots, {1, 1, 1}, {}});
  bool inplace = false;
  for (int64_t i = 0; i < count; ++i) {
    const lce_beam_state& st = states[i];
    if (st.segments < 0 || st.segments > kI32Max || st.segment_bytes < 0 ||
        st.segment_bytes > (int64_t(1) << 50))
      return LCE_ERR_BAD_SHAPE;
    if (st.segments == 0 || st.segment_bytes == 0) continue;
    if (!st.in || !st.out) return LCE_ERR_NULL_ARG;
    if (used.size() == 1) inplace = st.in == st.out;  // as the first state that holds something
    const int64_t bi = state_bytes(batch, beams, st.in_entry, st.in_beam, st.in_segment,
                                   st.segments, st.segment_bytes);
    const int64_t bo = state_bytes(batch, slots, st.out_entry, st.out_beam, st.out_segment,
                                   st.segments, st.segment_bytes);
    if (bi < 0 || bo < 0 ||
        !runs_apart(batch, slots, st.out_entry, st.out_beam, st.out_segment, st.segments,
                    st.segment_bytes) ||
        beam_reorder_groups(st, batch, beams, slots, inplace) > (int64_t(1) << 23))
      return LCE_ERR_BAD_SHAPE;
    const bool same = st.in == st.out && st.in_entry == st.out_entry &&
                      st.in_beam == st.out_beam && st.in_segment == st.out_segment &&
                      slots == beams;
    if (same != inplace) return LCE_ERR_OVERLAP;
    used.push_back({span(st.out, bo), true, st.segment_bytes, {batch, slots, st.segments},
                    {st.out_entry, st.out_beam, st.out_segment}});
    if (!inplace)
      used.push_back({span(st.in, bi), false, st.segment_bytes, {batch, beams, st.segments},
                      {st.in_entry, st.in_beam, st.in_segment}});
  }
  if (written_meets(used, open)) return LCE_ERR_OVERLAP;
  const int rc = check_device();
  if (rc != LCE_OK) return rc;
  LCE_TRY_HIP(beam_reorder_run(states, count, parents, batch, beams, slots, inplace,
                               static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

}  // extern "C"
