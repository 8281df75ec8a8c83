// Launch wrappers of the linear operators (internal; not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "linear_plan.hpp"

namespace moe {

struct LinearArgs {
  const void* a;       // columns' operand: kFwd, kDx: w; kDw: x
  const void* b;       // rows' operand: kFwd: x; kDx, kDw: dy
  const float* as;     // fp8 only: weight scales [groups, ceil(N/128), ceil(K/128)]
  const float* bs;     // fp8 only: row scales [rows, ceil(K/128)]
  const int32_t* off;  // [groups + 1], or nullptr: one group of all rows
  void* out;
  int rows, N, K, groups;
  void* part;          // workspace: f32 partial sums of a split reduction
  // with an epilogue (launch_linear_act)
  const void* bias = nullptr;  // [groups, N] of in_type, or none
  const void* res = nullptr;   // added to the result: [rows, N], gated [rows, N / 2], of out_type, or none
  void* pre = nullptr;         // receives the values before the activation, [rows, N] of out_type, or none
  int act = 0;
};

size_t linear_workspace(int rows, int N, int K, int groups, int in_type);
hipError_t launch_linear(int op, int in_type, int out_type, const LinearArgs& p, void* ws, hipStream_t st);

// The product with an epilogue (kernels_linear_act.hip): z = x w^T + bias, out =
// act(z) + res, gated: act(z[:, :N / 2]) z[:, N / 2:] + res.
hipError_t launch_linear_act_bf16(int out_type, bool gated, const LinearArgs& p, void* ws, hipStream_t st);
hipError_t launch_linear_act_f16(int out_type, bool gated, const LinearArgs& p, void* ws, hipStream_t st);

// The gradient through it (kernels_act_backward.hip): dz [rows, N] of in_type, db
// [groups, N] f32 or none, from dy [rows, N] (gated: N / 2) and pre [rows, N] of out_type.
struct ActBackwardArgs {
  const void *dy, *pre;
  const int32_t* off;
  void* dz;
  float* db;
  int rows, N, groups, act;
};
size_t act_backward_workspace(int rows, int N, int groups);
hipError_t launch_act_backward(int in_type, int out_type, bool gated, const ActBackwardArgs& p, void* ws, hipStream_t st);

// Sum of squares of tensors, and the tensors scaled (kernels_grad.hip).
struct GradTensor {
  const void* in;
  void* out;
  int64_t n;
  int type;  // kBF16, kF16, kF32
};
size_t grad_workspace(int count);
hipError_t launch_grad_norm(const GradTensor* t, int count, float* norm, void* ws, hipStream_t st);
hipError_t launch_grad_clip(const GradTensor* t, int count, float max_norm, float* norm, void* ws, hipStream_t st);

// fp8 codes and f32 scales per 128 columns of `rows` rows; swiglu: of
// silu(x[:, :K]) * x[:, K:].  ldx: elements between rows of x.
hipError_t launch_fp8_quant(const void* x, int x_type, bool swiglu, int rows, int K, int64_t ldx, uint8_t* q,
                            float* qs, hipStream_t st);

}  // namespace moe
