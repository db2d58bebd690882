// extern "C" entry points of the embedding, layer norm and vocabulary-piece operators: argument
// validation, all of it before any HIP call, then the launch code in embed_kernels.hip,
// norm_kernels.hip and flce_pieces.hip.
#include <limits>

#include "capi_checks.h"
#include "common.h"
#include "flce_pieces.h"
#include "lce_masked.h"
#include "ops.h"

namespace {

using namespace lce;

constexpr int64_t kI32Max = std::numeric_limits<int32_t>::max();

// Bytes of an element, 0 for an unknown type.
int64_t dtype_size(int dtype) {
  return dtype == LCE_DTYPE_BF16 || dtype == LCE_DTYPE_F16 ? 2 : dtype == LCE_DTYPE_F32 ? 4 : 0;
}

bool matrix_fits(int64_t rows, int64_t ld) {
  return !mul_overflows(rows, ld) && !mul_overflows(rows * ld, 4);
}

constexpr int64_t kThreadsMax = std::numeric_limits<uint32_t>::max();  // of one launch

int embed_check_shape(int64_t n, int64_t h, int64_t v) {
  return n < 0 || n > kI32Max || v < 1 || v > kI32Max || h < 1 || h > (int64_t(1) << 20)
             ? LCE_ERR_BAD_SHAPE
             : LCE_OK;
}
// The lookup takes a power of two of threads a row, 64 bytes each, where 256 of them hold it, and
// whole workgroups of 256.
bool lookup_fits(int64_t n, int64_t h, int64_t el) {
  return n * (h * el / 32 + 2) + 256 <= kThreadsMax;
}
// The gradient takes 8 threads a position to sort, 16 a table row to zero (where there are no
// positions one per 64 bytes, at most v * h / 16 + v / 4), and at most h + 512 per chunk of up
// to 512 positions to sum and join.
int embed_bwd_check_shape(int64_t n, int64_t h, int64_t v) {
  if (embed_check_shape(n, h, v) != LCE_OK) return LCE_ERR_BAD_SHAPE;
  return n > (int64_t(1) << 28) || v > (int64_t(1) << 27) || v * h > (int64_t(1) << 36) ||
                 (n == 0 && v * h > (int64_t(1) << 36) - (int64_t(1) << 30)) ||
                 n / 512 * (h + 512) > kThreadsMax / 2
             ? LCE_ERR_BAD_SHAPE
             : LCE_OK;
}

int norm_check_shape(int64_t n, int64_t h) {
  return n < 0 || n > kI32Max || h < 1 || h > LAYERNORM_MAX_H ? LCE_ERR_BAD_SHAPE : LCE_OK;
}

// The row limit keeps every byte offset inside one K slice of a 64-column panel below 2^32; the
// limits of classes and of 256 x 256 tiles the threads of a launch (4 a class where few rows are
// scored, 512 a tile).
int piece_check_shape(int64_t n, int64_t h, int64_t v) {
  if (n < 0 || n > (int64_t(1) << 23) || h < 1 || h % 8 != 0 || h > (int64_t(1) << 20) || v < 1 ||
      v > (int64_t(1) << 29) || (n + 255) / 256 * ((v + 255) / 256) >= (int64_t(1) << 23))
    return LCE_ERR_BAD_SHAPE;
  return LCE_OK;
}
int piece_check_vocab(int64_t v, int64_t v_start, int64_t vocab) {
  return vocab < 1 || vocab > kI32Max || v_start < 0 || v > vocab || v_start > vocab - v
             ? LCE_ERR_BAD_SHAPE
             : LCE_OK;
}

}  // namespace

extern "C" {

int embed_fwd(const void* weight, int dtype, int64_t v, int64_t h, int64_t ldw,
              const int32_t* tokens, int64_t n, int32_t ignore_index, float scale, void* out,
              int64_t ldo, int32_t* status_out, void* stream) {
  int rc = embed_check_shape(n, h, v);
  if (rc != LCE_OK) return rc;
  const int64_t el = dtype_size(dtype);
  if (!el) return LCE_ERR_BAD_DTYPE;
  if (ldw < h || ldo < h || !matrix_fits(v, ldw) || !matrix_fits(n, ldo) ||
      !lookup_fits(n, h, el))
    return LCE_ERR_BAD_SHAPE;
  if (!weight || (n > 0 && (!tokens || !out))) return LCE_ERR_NULL_ARG;
  if (!aligned(weight, el) || !aligned(out, el) || !aligned(tokens, 4) || !aligned(status_out, 4))
    return LCE_ERR_ALIGNMENT;
  {
    const Span wr[] = {span(out, matrix_bytes(n, ldo, h, el)), span(status_out, 4)};
    const Span rd[] = {span(weight, matrix_bytes(v, ldw, h, el)), span(tokens, 4 * n)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const EmbedFwdArgs a{weight, dtype, v, h, ldw, tokens, n, ignore_index, scale, out, ldo,
                       status_out};
  LCE_TRY_HIP(embed_fwd_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int embed_workspace_size(int64_t n, int64_t h, int64_t v, size_t* bytes) {
  if (!bytes) return LCE_ERR_NULL_ARG;
  const int rc = embed_bwd_check_shape(n, h, v);
  if (rc != LCE_OK) return rc;
  *bytes = embed_workspace_bytes(n, h);
  return LCE_OK;
}

int embed_bwd(const void* grad, int dtype, int64_t ldg, const int32_t* tokens, int64_t n,
              int64_t h, int64_t v, int32_t ignore_index, float scale, uint32_t flags,
              void* grad_weight, int grad_dtype, int64_t ldw, int32_t* status_out,
              void* workspace, size_t workspace_bytes, void* stream) {
  if (flags & ~EMBED_ACCUMULATE) return LCE_ERR_BAD_FLAGS;
  int rc = embed_bwd_check_shape(n, h, v);
  if (rc != LCE_OK) return rc;
  const int64_t el = dtype_size(dtype), wl = dtype_size(grad_dtype);
  if (!el || !wl || (grad_dtype != dtype && grad_dtype != LCE_DTYPE_F32)) return LCE_ERR_BAD_DTYPE;
  if (ldg < h || ldw < h || !matrix_fits(n, ldg) || !matrix_fits(v, ldw)) return LCE_ERR_BAD_SHAPE;
  if (!grad_weight || (n > 0 && (!tokens || !grad))) return LCE_ERR_NULL_ARG;
  const size_t need = embed_workspace_bytes(n, h);
  if (!workspace || workspace_bytes < need) return LCE_ERR_WORKSPACE;
  if (!aligned(grad, el) || !aligned(grad_weight, wl) || !aligned(tokens, 4) ||
      !aligned(status_out, 4) || !aligned(workspace, 256))
    return LCE_ERR_ALIGNMENT;
  {
    const Span wr[] = {span(workspace, int64_t(need)),
                       span(grad_weight, matrix_bytes(v, ldw, h, wl)), span(status_out, 4)};
    const Span rd[] = {span(grad, matrix_bytes(n, ldg, h, el)), span(tokens, 4 * n)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const EmbedBwdArgs a{grad, dtype, ldg, tokens, n, h, v, ignore_index, scale, flags,
                       grad_weight, grad_dtype, ldw, status_out, workspace};
  LCE_TRY_HIP(embed_bwd_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int layernorm_fwd(const void* x, int dtype, int64_t n, int64_t h, int64_t ldx, const void* weight,
                  const void* bias, int param_dtype, float eps, void* y, int64_t ldy,
                  float* mean_out, float* rstd_out, void* stream) {
  int rc = norm_check_shape(n, h);
  if (rc != LCE_OK) return rc;
  const int64_t el = dtype_size(dtype), pl = dtype_size(param_dtype);
  if (!el || !pl || (param_dtype != dtype && param_dtype != LCE_DTYPE_F32))
    return LCE_ERR_BAD_DTYPE;
  if (ldx < h || ldy < h || !matrix_fits(n, ldx) || !matrix_fits(n, ldy) || !(eps >= 0.f))
    return LCE_ERR_BAD_SHAPE;
  if (n > 0 && (!x || !y)) return LCE_ERR_NULL_ARG;
  if (!aligned(x, el) || !aligned(y, el) || !aligned(weight, pl) || !aligned(bias, pl) ||
      !aligned(mean_out, 4) || !aligned(rstd_out, 4))
    return LCE_ERR_ALIGNMENT;
  {
    const bool inplace = x == y && ldx == ldy;
    const Span wr[] = {span(y, matrix_bytes(n, ldy, h, el)), span(mean_out, 4 * n),
                       span(rstd_out, 4 * n)};
    const Span rd[] = {span(inplace ? nullptr : x, matrix_bytes(n, ldx, h, el)),
                       span(weight, pl * h), span(bias, pl * h)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const NormFwdArgs a{x, dtype, n, h, ldx, weight, bias, param_dtype, eps, y, ldy, mean_out,
                      rstd_out};
  LCE_TRY_HIP(layernorm_fwd_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int layernorm_workspace_size(int64_t n, int64_t h, size_t* bytes) {
  if (!bytes) return LCE_ERR_NULL_ARG;
  const int rc = norm_check_shape(n, h);
  if (rc != LCE_OK) return rc;
  *bytes = layernorm_workspace_bytes(n, h);
  return LCE_OK;
}

int layernorm_bwd(const void* grad, int dtype, int64_t ldg, const void* x, int64_t ldx,
                  const float* mean, const float* rstd, const void* weight, int param_dtype,
                  int64_t n, int64_t h, uint32_t flags, void* grad_x, int64_t lddx,
                  void* grad_weight, void* grad_bias, int grad_param_dtype, void* workspace,
                  size_t workspace_bytes, void* stream) {
  if (flags & ~LAYERNORM_ACCUMULATE) return LCE_ERR_BAD_FLAGS;
  int rc = norm_check_shape(n, h);
  if (rc != LCE_OK) return rc;
  const int64_t el = dtype_size(dtype), pl = dtype_size(param_dtype),
                gl = dtype_size(grad_param_dtype);
  if (!el || !pl || !gl || (param_dtype != dtype && param_dtype != LCE_DTYPE_F32) ||
      (grad_param_dtype != param_dtype && grad_param_dtype != LCE_DTYPE_F32))
    return LCE_ERR_BAD_DTYPE;
  if (ldg < h || ldx < h || (grad_x && lddx < h) || !matrix_fits(n, ldg) || !matrix_fits(n, ldx) ||
      (grad_x && !matrix_fits(n, lddx)))
    return LCE_ERR_BAD_SHAPE;
  if (n > 0 && (!grad || !x || !mean || !rstd)) return LCE_ERR_NULL_ARG;
  const bool params = grad_weight || grad_bias;
  const size_t need = params ? layernorm_workspace_bytes(n, h) : 0;
  if (params && (!workspace || workspace_bytes < need)) return LCE_ERR_WORKSPACE;
  if (!aligned(grad, el) || !aligned(x, el) || !aligned(grad_x, el) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(weight, pl) || !aligned(grad_weight, gl) ||
      !aligned(grad_bias, gl) || (params && !aligned(workspace, 256)))
    return LCE_ERR_ALIGNMENT;
  {
    const bool inplace = grad == grad_x && ldg == lddx;
    const Span wr[] = {span(params ? workspace : nullptr, int64_t(need)),
                       span(grad_x, grad_x ? matrix_bytes(n, lddx, h, el) : 0),
                       span(grad_weight, gl * h), span(grad_bias, gl * h)};
    const Span rd[] = {span(inplace ? nullptr : grad, matrix_bytes(n, ldg, h, el)),
                       span(x, matrix_bytes(n, ldx, h, el)), span(mean, 4 * n),
                       span(rstd, 4 * n), span(weight, pl * h)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const NormBwdArgs a{grad, dtype, ldg, x, ldx, mean, rstd, weight, param_dtype, n, h, flags,
                      grad_x, lddx, grad_weight, grad_bias, grad_param_dtype, workspace};
  LCE_TRY_HIP(layernorm_bwd_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int flce_piece_fwd_workspace_size(int64_t n, int64_t h, int64_t v, size_t* bytes) {
  if (!bytes) return LCE_ERR_NULL_ARG;
  const int rc = piece_check_shape(n, h, v);
  if (rc != LCE_OK) return rc;
  *bytes = piece_fwd_workspace_bytes(n, h, v);
  return LCE_OK;
}

int flce_piece_loss_workspace_size(int64_t n, size_t* bytes) {
  if (!bytes) return LCE_ERR_NULL_ARG;
  const int rc = piece_check_shape(n, 8, 1);
  if (rc != LCE_OK) return rc;
  *bytes = piece_loss_workspace_bytes(n);
  return LCE_OK;
}

int flce_piece_bwd_workspace_size(int64_t n, int64_t h, int64_t v, size_t* bytes) {
  if (!bytes) return LCE_ERR_NULL_ARG;
  const int rc = piece_check_shape(n, h, v);
  if (rc != LCE_OK) return rc;
  *bytes = piece_bwd_workspace_bytes(n, h, v);
  return LCE_OK;
}

int flce_piece_fwd(const uint16_t* hidden, const uint16_t* weight, const float* bias,
                   const int32_t* labels, int64_t n, int64_t h, int64_t v, int64_t v_start,
                   int64_t vocab, int32_t ignore_index, uint32_t flags, float* state,
                   void* workspace, size_t workspace_bytes, void* stream) {
  if (flags & ~FLCE_PIECE_FIRST) return LCE_ERR_BAD_FLAGS;
  int rc = piece_check_shape(n, h, v);
  if (rc != LCE_OK || (rc = piece_check_vocab(v, v_start, vocab)) != LCE_OK) return rc;
  if (!weight || (n > 0 && (!hidden || !labels || !state))) return LCE_ERR_NULL_ARG;
  const size_t need = piece_fwd_workspace_bytes(n, h, v);
  if (!workspace || workspace_bytes < need) return LCE_ERR_WORKSPACE;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(bias, 4) || !aligned(labels, 4) ||
      !aligned(state, 4) || !aligned(workspace, 256))
    return LCE_ERR_ALIGNMENT;
  {
    const Span wr[] = {span(workspace, int64_t(need)), span(state, 12 * n)};
    const Span rd[] = {span(hidden, 2 * n * h), span(weight, 2 * v * h), span(bias, 4 * v),
                       span(labels, 4 * n)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const PieceFwdArgs a{hidden, weight, bias, labels, n, h, v, v_start, vocab, ignore_index, flags,
                       state, workspace};
  LCE_TRY_HIP(piece_fwd_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int flce_piece_loss(const float* state, const int32_t* labels, int64_t n, int64_t vocab,
                    int32_t ignore_index, int64_t num_label_tokens, float* loss_out,
                    float* lse_out, float* row_loss_out, int32_t* status_out, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int rc = piece_check_shape(n, 8, 1);
  if (rc != LCE_OK || (rc = piece_check_vocab(1, 0, vocab)) != LCE_OK) return rc;
  if (n > 0 && (!state || !labels)) return LCE_ERR_NULL_ARG;
  const size_t need = piece_loss_workspace_bytes(n);
  if (!workspace || workspace_bytes < need) return LCE_ERR_WORKSPACE;
  if (!aligned(state, 4) || !aligned(labels, 4) || !aligned(loss_out, 4) || !aligned(lse_out, 4) ||
      !aligned(row_loss_out, 4) || !aligned(status_out, 4) || !aligned(workspace, 256))
    return LCE_ERR_ALIGNMENT;
  {
    const Span wr[] = {span(workspace, int64_t(need)), span(loss_out, 4), span(lse_out, 4 * n),
                       span(row_loss_out, 4 * n), span(status_out, 4)};
    const Span rd[] = {span(state, 12 * n), span(labels, 4 * n)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const PieceLossArgs a{state, labels, n, vocab, ignore_index, num_label_tokens, loss_out,
                        lse_out, row_loss_out, status_out, workspace};
  LCE_TRY_HIP(piece_loss_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

int flce_piece_bwd(const uint16_t* hidden, const uint16_t* weight, const float* bias,
                   const int32_t* labels, const float* lse, int64_t n, int64_t h, int64_t v,
                   int64_t v_start, int64_t vocab, int32_t ignore_index,
                   int64_t num_label_tokens, uint32_t flags, const float* grad_output,
                   const float* grad_rows, float* hidden_acc, uint16_t* grad_hidden,
                   void* grad_weight, int grad_weight_dtype, float* grad_bias, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (flags & ~(FLCE_PIECE_FIRST | FLCE_PIECE_LAST | FLCE_PIECE_ACCUMULATE))
    return LCE_ERR_BAD_FLAGS;
  int rc = piece_check_shape(n, h, v);
  if (rc != LCE_OK || (rc = piece_check_vocab(v, v_start, vocab)) != LCE_OK) return rc;
  if (grad_weight && grad_weight_dtype != LCE_DTYPE_BF16 && grad_weight_dtype != LCE_DTYPE_F32)
    return LCE_ERR_BAD_DTYPE;
  const bool first = flags & FLCE_PIECE_FIRST, last = flags & FLCE_PIECE_LAST;
  if (!weight || (n > 0 && (!hidden || !labels || !lse)) || (grad_bias && !bias) ||
      (grad_hidden && !hidden_acc && !(first && last)))
    return LCE_ERR_NULL_ARG;
  const size_t need = piece_bwd_workspace_bytes(n, h, v);
  if (!workspace || workspace_bytes < need) return LCE_ERR_WORKSPACE;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(bias, 4) || !aligned(labels, 4) ||
      !aligned(lse, 4) || !aligned(grad_output, 4) || !aligned(grad_rows, 4) ||
      !aligned(hidden_acc, 16) || !aligned(grad_hidden, 16) || !aligned(grad_weight, 16) ||
      !aligned(grad_bias, 4) || !aligned(workspace, 256))
    return LCE_ERR_ALIGNMENT;
  {
    const int64_t wl = grad_weight_dtype == LCE_DTYPE_F32 ? 4 : 2;
    const Span wr[] = {span(workspace, int64_t(need)), span(hidden_acc, 4 * n * h),
                       span(grad_hidden, 2 * n * h), span(grad_weight, wl * v * h),
                       span(grad_bias, 4 * v)};
    const Span rd[] = {span(hidden, 2 * n * h), span(weight, 2 * v * h), span(bias, 4 * v),
                       span(labels, 4 * n), span(lse, 4 * n), span(grad_output, 4),
                       span(grad_rows, 4 * n)};
    if ((rc = check_disjoint(wr, rd)) != LCE_OK) return rc;
  }
  if ((rc = check_device()) != LCE_OK) return rc;
  const PieceBwdArgs a{hidden, weight, bias, labels, lse, n, h, v, v_start, vocab, ignore_index,
                       num_label_tokens >= 0 ? num_label_tokens : -1, flags, grad_output,
                       grad_rows, hidden_acc, grad_hidden, grad_weight, grad_weight_dtype,
                       grad_bias, workspace};
  LCE_TRY_HIP(piece_bwd_run(a, static_cast<hipStream_t>(stream)));
  return LCE_OK;
}

}  // extern "C"
