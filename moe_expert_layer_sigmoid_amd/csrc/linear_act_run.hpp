// Launches of the products with an epilogue, for one operand type (two
// translation units, which build side by side).
#pragma once

#include <hip/hip_runtime.h>

#include "linear_kernel.hpp"

namespace moe {
namespace {

template <class C, int EP>
hipError_t run_shape(const LinearArgs& p, const Plan& pl, hipStream_t st) {
  const long blocks = (long)ceil_div(pl.nca * pl.nrb * pl.splits, kXcd) * kXcd;
  k_linear<C, EP><<<dim3((unsigned)blocks), C::KS * C::W * 64, 0, st>>>(p, pl);
  return hipGetLastError();
}

template <int IN, int EP>
hipError_t run_ep(int out_type, LinearArgs p, void* ws, hipStream_t st) {
  constexpr int OP = kFwd, G = EP == kGated ? 2 : 1;
  const bool big = streams(IN, p.rows, p.N, p.K, p.groups);
  if (few_rows(p.rows, p.N / G, p.groups)) {
    const dim3 grid((unsigned)ceil_div(p.N / G, 16), p.groups);
    if (big) k_linear_few<IN, true, EP><<<grid, kFewWaves * 64, 0, st>>>(p, out_type);
    else k_linear_few<IN, false, EP><<<grid, kFewWaves * 64, 0, st>>>(p, out_type);
    return hipGetLastError();
  }
  // (a gated tile of TA columns makes TA / 2 outputs: as many tiles as the plain product's)
  Choice c = choose(OP, IN, p.rows, p.N, p.K, p.groups);
  c.plan.out_type = out_type;
  c.plan.big = big;
  p.part = ws;
  hipError_t e;
  if (c.shape == 0) e = run_shape<Shape<IN, OP, 256, 256, 2, 4, 1, 2, 1>, EP>(p, c.plan, st);
  else if (c.shape == 1) e = run_shape<Shape<IN, OP, 256, 128, 4, 2, 1, 3, 1>, EP>(p, c.plan, st);
  else if (c.shape == 2) e = run_shape<Shape<IN, OP, 128, 128, 2, 2, 1, 2, 2>, EP>(p, c.plan, st);
  else if (c.shape == 3) e = run_shape<Shape<IN, OP, 128, 64, 2, 2, 1, 3, 2>, EP>(p, c.plan, st);
  else if (c.shape == 4) e = run_shape<Shape<IN, OP, 128, 64, 2, 2, 2, 3, 1>, EP>(p, c.plan, st);
  else if (c.shape == 5) e = run_shape<Shape<IN, OP, 128, 32, 2, 2, 1, 3, 2>, EP>(p, c.plan, st);
  else e = run_shape<Shape<IN, OP, 256, 192, 2, 4, 1, 2, 1>, EP>(p, c.plan, st);
  if (e != hipSuccess || c.plan.splits == 1) return e;
  const size_t want = ((size_t)p.rows * ceil_div(p.N / G, 4) + 255) / 256;
  const unsigned blocks = (unsigned)(want < 2048 ? want : 2048);
  if (out_type == kF32) k_linear_join_act<kF32, IN, EP><<<blocks, 256, 0, st>>>(p, c.plan.splits);
  else k_linear_join_act<IN, IN, EP><<<blocks, 256, 0, st>>>(p, c.plan.splits);
  return hipGetLastError();
}

template <int IN>
hipError_t run_act(int out_type, bool gated, const LinearArgs& p, void* ws, hipStream_t st) {
  return gated ? run_ep<IN, kGated>(out_type, p, ws, st) : run_ep<IN, kAct>(out_type, p, ws, st);
}

}  // namespace
}  // namespace moe
