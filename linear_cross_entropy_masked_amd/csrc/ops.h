// Internal interface of the embedding (embed_kernels.hip) and layer norm (norm_kernels.hip)
// operators, between their C-ABI entry points and their launch code.
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

}  // namespace lce
