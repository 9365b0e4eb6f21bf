// Launchers of the training-step operators (include/bmoe_norm.h,
// include/bmoe_update.h).
#pragma once

#include "common.hpp"

namespace bmoe {

// Layer norm (layer_norm.hip).
struct LnFwdArgs {
  const void* x;            // [rows][width]
  const void* res;          // [rows][width] or null
  const float* gamma;       // [width] or null
  const float* beta;        // [width] or null
  void* sum;                // [rows][width] when res is set
  void* y;                  // [rows][width]
  float* mean;              // [rows] or null
  float* rstd;              // [rows] when mean is set
  float eps;
  int32_t rows, width;
};
struct LnBwdArgs {
  const void* dy;           // [rows][width], its own dtype
  const void* s;            // [rows][width]
  const float* gamma;       // [width] or null
  const float* mean;        // [rows]
  const float* rstd;        // [rows]
  const void* d_sum;        // [rows][width] or null
  void* dx;                 // [rows][width]
  float* dgamma;            // [width] or null
  float* dbeta;             // [width] when dgamma is set
  float* part;              // the workspace
  int32_t rows, width;
  int32_t row_blocks;       // the launcher's
};
size_t ln_bwd_workspace(int rows, int width);
hipError_t launch_ln_fwd(const LnFwdArgs& a, int act, hipStream_t s);
hipError_t launch_ln_bwd(LnBwdArgs a, int act, int dact, hipStream_t s);

// Latent substrate step and ternary codes (substrate_step.hip).
struct SubStepArgs {
  const float* w;           // [n]
  const uint16_t* o;        // [n] bf16 or null
  float* w_out;             // [n] when o is set
  uint32_t* packed;         // [n / 16]
  float* scale;             // 1 or null
  double* part;             // sub_step_blocks partial sums
  double step, keep;        // W' = keep W - step O
  size_t n;                 // weights, a multiple of 16
};
size_t sub_step_workspace(size_t n);
hipError_t launch_sub_step(const SubStepArgs& a, hipStream_t s);

// Orthogonalised update (orthogonalize.hip).
struct OrthoArgs {
  const void* grad;         // [rows][cols]
  const float* m;           // [rows][cols] or null
  float* m_out;             // [rows][cols] when m is set
  uint16_t* out;            // [rows][cols] bf16
  float mu;
  int32_t rows, cols, nesterov, grad_bf16;
  void* ws;
};
size_t ortho_workspace(int rows, int cols);
hipError_t launch_orthogonalize(const OrthoArgs& a, hipStream_t s);

}  // namespace bmoe
