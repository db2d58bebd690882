// Internal interface of the linear cross entropy in pieces of the vocabulary (flce_pieces.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lce {

struct PieceFwdArgs {
  const uint16_t* hidden;
  const uint16_t* weight;
  const float* bias;
  const int32_t* labels;
  int64_t n, h, v, v_start, vocab;
  int32_t ignore_index;
  uint32_t flags;
  float* state;
  void* workspace;
};
size_t piece_fwd_workspace_bytes(int64_t n, int64_t h, int64_t v);
hipError_t piece_fwd_run(const PieceFwdArgs& a, hipStream_t s);

struct PieceLossArgs {
  const float* state;
  const int32_t* labels;
  int64_t n, vocab;
  int32_t ignore_index;
  int64_t num_label_tokens;
  float *loss_out, *lse_out, *row_loss_out;
  int32_t* status_out;
  void* workspace;
};
size_t piece_loss_workspace_bytes(int64_t n);
hipError_t piece_loss_run(const PieceLossArgs& a, hipStream_t s);

struct PieceBwdArgs {
  const uint16_t* hidden;
  const uint16_t* weight;
  const float* bias;
  const int32_t* labels;
  const float* lse;
  int64_t n, h, v, v_start, vocab;
  int32_t ignore_index;
  int64_t num_label_tokens;
  uint32_t flags;
  const float* grad_output;
  const float* grad_rows;
  float* hidden_acc;
  uint16_t* grad_hidden;
  void* grad_weight;
  int grad_weight_dtype;
  float* grad_bias;
  void* workspace;
};
size_t piece_bwd_workspace_bytes(int64_t n, int64_t h, int64_t v);
hipError_t piece_bwd_run(const PieceBwdArgs& a, hipStream_t s);

}  // namespace lce
