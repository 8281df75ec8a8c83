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
};

size_t linear_workspace(int rows, int N, int K, int groups, int in_type);
hipError_t launch_linear(int op, int in_type, int out_type, const LinearArgs& p, void* ws, hipStream_t st);

// fp8 codes and f32 scales per 128 columns of `rows` rows; swiglu: of
// silu(x[:, :K]) * x[:, K:].  ldx: elements between rows of x.
hipError_t launch_fp8_quant(const void* x, int x_type, bool swiglu, int rows, int K, int64_t ldx, uint8_t* q,
                            float* qs, hipStream_t st);

}  // namespace moe
