// Launch wrappers of the linear operators (internal; not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// moe_dtype_t of include/moe.h
enum { kBF16 = 0, kF16 = 1, kF32 = 2, kFP8 = 3 };

// What a product computes; "columns" are the output's contiguous dimension.
//  kFwd: y[row, n]  = sum_k x[row, k] w[g, n, k]
//  kDx:  dx[row, k] = sum_n dy[row, n] w[g, n, k]
//  kDw:  dw[g, n, k] = sum over the group's rows of dy[row, n] x[row, k]
enum { kFwd = 0, kDx = 1, kDw = 2 };

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
