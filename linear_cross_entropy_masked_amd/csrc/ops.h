// Internal interface of the embedding (embed_kernels.hip), norm (norm_kernels.hip, rms_kernels.hip),
// 8-bit product (fp8_kernels.hip) and beam search (beam_kernels.hip) operators, between their
// C-ABI entry points and their launch code.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lce_masked.h"

namespace lce {

struct EmbedFwdArgs {
  const void* weight;
  int dtype;
  int64_t v, h, ldw;
  const int32_t* tokens;
  int64_t n;
  int32_t ignore_index;
  float scale;
  void* out;
  int64_t ldo;
  int32_t* status_out;
};
hipError_t embed_fwd_run(const EmbedFwdArgs& a, hipStream_t s);

struct EmbedBwdArgs {
  const void* grad;
  int dtype;
  int64_t ldg;
  const int32_t* tokens;
  int64_t n, h, v;
  int32_t ignore_index;
  float scale;
  uint32_t flags;
  void* grad_weight;
  int grad_dtype;
  int64_t ldw;
  int32_t* status_out;
  void* workspace;
};
size_t embed_workspace_bytes(int64_t n, int64_t h);
hipError_t embed_bwd_run(const EmbedBwdArgs& a, hipStream_t s);
// The same of bf16 rows, where row i counts coef[i] times and a sum, rounded to bf16 whatever the
// table's type, *scale times (NULL: a.scale times). Rows of grad_weight that no position names are
// left as they are; bit v of named (NULL: not) is set for the others. `sorted`: the order is there
// already, each position's token and row where embed_weighted_order() says, tokens that carry no row
// being v.
size_t embed_weighted_workspace_bytes(int64_t n, int64_t h);
void embed_weighted_order(void* workspace, int64_t n, int64_t h, int32_t** tokens, int32_t** rows);
hipError_t embed_weighted_run(const EmbedBwdArgs& a, const float* coef, const float* scale,
                              bool sorted, uint32_t* named, hipStream_t s);

struct NormFwdArgs {
  const void* x;
  int dtype;
  int64_t n, h, ldx;
  const void* weight;
  const void* bias;
  int param_dtype;
  float eps;
  void* y;
  int64_t ldy;
  float* mean_out;
  float* rstd_out;
};
hipError_t layernorm_fwd_run(const NormFwdArgs& a, hipStream_t s);

struct NormBwdArgs {
  const void* grad;
  int dtype;
  int64_t ldg;
  const void* x;
  int64_t ldx;
  const float* mean;
  const float* rstd;
  const void* weight;
  int param_dtype;
  int64_t n, h;
  uint32_t flags;
  void* grad_x;
  int64_t lddx;
  void* grad_weight;
  void* grad_bias;
  int grad_param_dtype;
  void* workspace;
};
size_t layernorm_workspace_bytes(int64_t n, int64_t h);
hipError_t layernorm_bwd_run(const NormBwdArgs& a, hipStream_t s);

// Root-mean-square norm (rms_kernels.hip); scales: 8-bit outputs.
struct RmsFwdArgs {
  const void* x;
  int dtype;
  int64_t n, h, ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  int param_dtype;
  float eps;
  void* y;
  int64_t ldy;
  void* residual_out;
  int64_t ldro;
  float* rstd_out;
  void* scales;
  int scale_dtype;
  int64_t lds;
};
hipError_t rmsnorm_fwd_run(const RmsFwdArgs& a, hipStream_t s);

struct RmsBwdArgs {
  const void* grad;
  int dtype;
  int64_t ldg;
  const void* x;
  int64_t ldx;
  const float* rstd;
  const void* weight;
  int param_dtype;
  const void* grad_residual;
  int64_t ldgr, n, h;
  uint32_t flags;
  void* grad_x;
  int64_t lddx;
  void* grad_weight;
  int grad_param_dtype;
  void* workspace;
};
size_t rmsnorm_workspace_bytes(int64_t n, int64_t h);
hipError_t rmsnorm_bwd_run(const RmsBwdArgs& a, hipStream_t s);

// 8-bit blocks and their product (fp8_kernels.hip).
struct Fp8QuantizeArgs {
  const void* x;
  int dtype;
  int64_t n, h, ldx, block_rows;
  uint8_t* q;
  int64_t ldq;
  void* scales;
  int scale_dtype;
  int64_t lds;
};
int64_t fp8_quantize_groups(int64_t n, int64_t h, int64_t block_rows);  // workgroups
hipError_t fp8_quantize_run(const Fp8QuantizeArgs& a, hipStream_t s);

struct Fp8MatmulArgs {
  const uint8_t* a;
  int64_t lda;
  const void* a_scales;
  int64_t ldas;
  const uint8_t* b;
  int64_t ldb;
  const void* b_scales;
  int64_t ldbs;
  int scale_dtype;
  const float* bias;
  int64_t m, n, k;
  void* out;
  int out_dtype;
  int64_t ldo;
  void* workspace;
  bool precise;  // fp32 sums whatever the output's type
};
size_t fp8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k);
hipError_t fp8_matmul_run(const Fp8MatmulArgs& a, hipStream_t s);

// A beam search's step (beam_kernels.hip).
struct BeamStepArgs {
  const void* logits;
  int dtype;
  int64_t batch, beams, v, ldl;
  const float* scores;
  const uint8_t* finished;
  int32_t eos;
  int64_t num;
  int32_t ignore_index;
  float* scores_out;
  int32_t* parents_out;
  int32_t* tokens_out;
  uint8_t* finished_out;
  int32_t* status_out;
  void* workspace;
};
int64_t beam_step_slices(int64_t rows, int64_t v);  // workgroups over the logits
size_t beam_step_workspace_bytes(int64_t batch, int64_t beams, int64_t v, int64_t num);
hipError_t beam_step_run(const BeamStepArgs& a, hipStream_t s);

// Workgroups of one state's reordering.
int64_t beam_reorder_groups(const lce_beam_state& st, int64_t batch, int64_t beams, int64_t slots,
                            bool inplace);
hipError_t beam_reorder_run(const lce_beam_state* states, int64_t count, const int32_t* parents,
                            int64_t batch, int64_t beams, int64_t slots, bool inplace,
                            hipStream_t s);

}  // namespace lce
