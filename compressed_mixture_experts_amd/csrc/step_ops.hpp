// Launchers of the training-step operators (include/bmoe_norm.h,
// include/bmoe_update.h, include/bmoe_adamw.h, include/bmoe_block.h,
// include/bmoe_ffn.h).
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

// AdamW (adamw.hip).
enum AwFlags { AW_GRAD_BF16 = 1, AW_EIGHT = 2, AW_ALIGNED = 4 };
constexpr int AW_TENSORS = 40;  // of a launch
struct AwTensor {
  float* p;                 // [n]
  const void* g;            // [n]
  void* m;                  // [n] fp32 or codes
  void* v;
  uint8_t* me;              // a byte a block of 256 with codes
  uint8_t* ve;
  uint16_t* copy;           // [n] bf16 or null
  int64_t n;
  float lr_scale, decay;
  uint32_t index;           // the tensor's place in the call
  uint32_t flags;
};
struct AwScalars {
  float beta1, rest1, beta2, rest2, eps;   // rest = 1 - beta
  float lr;
  float by1, root2;         // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  double log1, log2;        // log(beta)
  int64_t step;
  const int64_t* step_device;
  const float* lr_device;
  const float* grad_scale;
  uint32_t seed;
};
// count_up: raised by 1 first, or null
hipError_t launch_adamw(const AwTensor* tensors, int count, const AwScalars& s, int64_t* count_up, hipStream_t stream);
// codes' values: of m to p and of v to copy (arrays of the given type, null: not wanted)
hipError_t launch_adamw_values(const AwTensor* tensors, int count, bool bf16, hipStream_t stream);

// Norms around a block (block_norm.hip).
enum BnGate { BN_GATE_NONE = 0, BN_GATE_CHANNEL = 1, BN_GATE_ROWS = 2 };
struct BnFwdArgs {
  const void* b;            // [rows][width]
  const void* r;            // [rows][width] or null
  const void* gate;         // [width] fp32, [rows][width] or null
  const float* gamma_post;  // [width] or null, as the next three
  const float* beta_post;
  const float* gamma;
  const float* beta;
  void* s;                  // [rows][width]
  void* y;                  // [rows][width]
  float4* stats;            // [rows] or null
  float alpha, scale, eps;
  int32_t rows, width, layer, post, gate_kind;
};
struct BnBwdArgs {
  const void* dy;           // [rows][width], its own dtype
  const void* b;            // [rows][width]
  const void* s;            // [rows][width]
  const float4* stats;      // [rows]
  const void* d_sum;        // [rows][width] or null
  const void* gate;         // as in the forward
  const float* gamma_post;
  const float* beta_post;
  const float* gamma;
  void* db;                 // [rows][width]
  void* dr;                 // [rows][width] or null
  void* d_gate;             // [rows][width] with a gate of rows, or null
  float* d_gamma_post;      // [width] or null, as the next four
  float* d_beta_post;
  float* d_gate_channel;
  float* d_gamma;
  float* d_beta;
  float* part;              // the workspace, null without any of those five
  float alpha, scale;
  int32_t rows, width, layer, post, gate_kind;
};
size_t bn_bwd_workspace(int rows, int width);
hipError_t launch_block_norm_fwd(const BnFwdArgs& a, int act, hipStream_t s);
hipError_t launch_block_norm_bwd(const BnBwdArgs& a, int act, int dact, hipStream_t s);

// Dense gated feed-forward block (gated_ffn.hip), bf16.
struct GfFwdArgs {
  const uint16_t* x;        // [tokens][d]
  const uint16_t* w_in;     // [2 ff][d]
  const uint16_t* w_down;   // [d][ff]
  const uint16_t* add;      // [tokens][d] or null
  uint16_t* y;              // [tokens][d]
  uint16_t* state;          // [tokens][2 ff], [tokens][ff], then bytes [tokens][ff]; or null
  void* ws;
  int32_t tokens, d, ff, gelu;
};
struct GfBwdArgs {
  const uint16_t* x;
  const uint16_t* w_in;
  const uint16_t* w_down;
  const uint16_t* dy;       // [tokens][d]
  const uint16_t* state;
  const float* dx_add;      // [tokens][d] or null
  uint16_t* dx;             // [tokens][d] or null
  uint16_t* dw_in;          // [2 ff][d] or null
  uint16_t* dw_down;        // [d][ff] or null
  void* ws;
  int32_t tokens, d, ff;
};
size_t gf_forward_workspace(int tokens, int d, int ff, bool with_state);
size_t gf_backward_workspace(int tokens, int d, int ff);
hipError_t launch_gated_ffn_forward(const GfFwdArgs& a, hipStream_t s);
hipError_t launch_gated_ffn_backward(const GfBwdArgs& a, hipStream_t s);
// Which kernels those launch (bmoe_debug.h's numbers, in its order).
struct GfPlan {
  int32_t few, gate, y, y_shares, grad, joint, joint_parts, last[3], last_shares[3];
};
GfPlan gated_ffn_plan(int tokens, int d, int ff);

}  // namespace bmoe
