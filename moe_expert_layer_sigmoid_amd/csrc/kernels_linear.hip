// Linear operators on gfx950's matrix instructions: the fp8 product with a
// scale per block of 128, and the 16-bit products grouped by expert, forward
// and both gradients.
//
// One kernel template over the operand types and the three products.  The
// output's contiguous dimension ("columns") is the MFMA's A side, so that a
// lane holds four consecutive columns of one row; its rows are the B side.
//   y[row, n]   : A = w  [n][k],  B = x [row][k],   reduced over k
//   dx[row, k]  : A = w  [n][k]^T, B = dy [row][n], reduced over n
//   dw[n, k]    : A = x  [row][k]^T, B = dy [row][n]^T, reduced over rows
// An operand whose reduction is not contiguous is read from LDS with the
// transposing load.  fp8: the scales of a 128-column stage are constant over it, so
// one 16x16x128 product per tile is scaled by xs * ws in f32 and added to an
// f32 accumulator.
//
// Bound by the staging into LDS nearly everywhere (us, and with the products
// left out): fp8 8192 x 4096 x 7168 207 (2.3 PFLOP/s) and 182; 48 fp8 experts at
// 6144 rows 191 and 183; 48 bf16 experts 630 and 630 (5 TB/s past L2); 512 fp8
// rows 23 and 21.  With few rows an expert the weights stream at 6.9 TB/s.

#include <hip/hip_runtime.h>

#include "linear_kernel.hpp"

namespace moe {
namespace {

template <class C>
hipError_t run_shape(const LinearArgs& p, const Plan& pl, hipStream_t st) {
  long blocks;
  if (C::OP == kDw) blocks = (long)p.groups * (ceil_div(pl.nca * pl.nrb * pl.splits, kXcd) * kXcd);
  else blocks = (long)ceil_div(pl.nca * pl.nrb * pl.splits, kXcd) * kXcd;
  k_linear<C><<<dim3((unsigned)blocks), C::KS * C::W * 64, 0, st>>>(p, pl);
  return hipGetLastError();
}

template <int IN, int OP>
hipError_t run_op(int out_type, LinearArgs p, void* ws, hipStream_t st) {
  const bool big = streams(IN, p.rows, p.N, p.K, p.groups);
  if constexpr (OP == kFwd) {
    if (few_rows(p.rows, p.N, p.groups)) {
      const dim3 grid((unsigned)ceil_div(p.N, 16), p.groups);
      if (big) k_linear_few<IN, true><<<grid, kFewWaves * 64, 0, st>>>(p, out_type);
      else k_linear_few<IN, false><<<grid, kFewWaves * 64, 0, st>>>(p, out_type);
      return hipGetLastError();
    }
  }
  Choice c = choose(OP, IN, p.rows, p.N, p.K, p.groups);
  c.plan.out_type = out_type;
  c.plan.big = big;
  p.part = ws;
  hipError_t e;
  if (c.shape == 0) e = run_shape<Shape<IN, OP, 256, 256, 2, 4, 1, 2, 1>>(p, c.plan, st);
  else if (c.shape == 1) e = run_shape<Shape<IN, OP, 256, 128, 4, 2, 1, 3, 1>>(p, c.plan, st);
  else if (c.shape == 2) e = run_shape<Shape<IN, OP, 128, 128, 2, 2, 1, 2, 2>>(p, c.plan, st);
  else if (c.shape == 3) e = run_shape<Shape<IN, OP, 128, 64, 2, 2, 1, 3, 2>>(p, c.plan, st);
  else if (c.shape == 4) e = run_shape<Shape<IN, OP, 128, 64, 2, 2, 2, 3, 1>>(p, c.plan, st);
  else if (c.shape == 5) e = run_shape<Shape<IN, OP, 128, 32, 2, 2, 1, 3, 2>>(p, c.plan, st);
  else if constexpr (OP != kDw) e = run_shape<Shape<IN, OP, 256, 192, 2, 4, 1, 2, 1>>(p, c.plan, st);
  else return hipErrorInvalidValue;  // choose() does not take it for kDw
  if (e != hipSuccess || c.plan.splits == 1) return e;
  const int cols = OP == kFwd ? p.N : p.K;
  const int rows = OP == kDw ? p.groups * p.N : p.rows;  // a split output is at most kPartMax
  const size_t want = ((size_t)rows * ceil_div(cols, 4) + 255) / 256;
  const unsigned blocks = (unsigned)(want < 2048 ? want : 2048);
  if (out_type == kBF16) k_linear_join<kBF16><<<blocks, 256, 0, st>>>(p, rows, cols, c.plan.splits, OP != kDw);
  else if (out_type == kF16) k_linear_join<kF16><<<blocks, 256, 0, st>>>(p, rows, cols, c.plan.splits, OP != kDw);
  else k_linear_join<kF32><<<blocks, 256, 0, st>>>(p, rows, cols, c.plan.splits, OP != kDw);
  return hipGetLastError();
}

template <int IN>
hipError_t run_in(int op, int out_type, const LinearArgs& p, void* ws, hipStream_t st) {
  if (op == kFwd) return run_op<IN, kFwd>(out_type, p, ws, st);
  if (op == kDx) return run_op<IN, kDx>(out_type, p, ws, st);
  return run_op<IN, kDw>(out_type, p, ws, st);
}

}  // namespace

size_t linear_workspace(int rows, int N, int K, int groups, int in_type) {
  size_t n = part_bytes(kFwd, rows, N, K, groups);
  if (in_type != kFP8)
    for (int op = kDx; op <= kDw; ++op) {
      const size_t m = part_bytes(op, rows, N, K, groups);
      n = m > n ? m : n;
    }
  return n;
}

hipError_t launch_linear(int op, int in_type, int out_type, const LinearArgs& p, void* ws, hipStream_t st) {
  if (in_type == kFP8) return run_op<kFP8, kFwd>(out_type, p, ws, st);
  return in_type == kBF16 ? run_in<kBF16>(op, out_type, p, ws, st) : run_in<kF16>(op, out_type, p, ws, st);
}

}  // namespace moe
