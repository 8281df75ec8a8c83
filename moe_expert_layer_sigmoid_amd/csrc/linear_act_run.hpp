// Launches of the products with an epilogue, for one operand type (two
// translation units, which build side by side).
#pragma once

#include <hip/hip_runtime.h>

#include "linear_rows.hpp"

namespace moe {
namespace {

template <class C, int EP>
hipError_t run_shape(const LinearArgs& p, const Plan& pl, hipStream_t st) {
  const long blocks = (long)ceil_div(pl.nca * pl.nrb * pl.splits, kXcd) * kXcd;
  k_linear<C, EP><<<dim3((unsigned)blocks), C::KS * C::W * 64, 0, st>>>(p, pl);
  return hipGetLastError();
}

template <int IN, int EP>
hipError_t run_rows(int out_type, const LinearArgs& p, bool big, hipStream_t st) {
  const int live = p.rows < p.groups ? p.rows : p.groups;
  const long cols = (long)live * (p.N / (EP == kGated ? 2 : 1)), shares = (cols + kRowsLeastCols - 1) / kRowsLeastCols;
  const auto launch = [&](auto w) {
    constexpr int W = decltype(w)::value, kMost = 2 * kCus * kRingWaves / W;
    const unsigned blocks = (unsigned)(shares < kMost ? shares : kMost);
    if (big) k_linear_rows<IN, EP, true, W><<<blocks, W * 64, 0, st>>>(p, out_type);
    else k_linear_rows<IN, EP, false, W><<<blocks, W * 64, 0, st>>>(p, out_type);
  };
  if (cols <= 16 * kCus) launch(std::integral_constant<int, 8>{});
  else launch(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

template <int IN, int EP>
hipError_t run_ep(int out_type, LinearArgs p, void* ws, hipStream_t st) {
  constexpr int OP = kFwd, G = EP == kGated ? 2 : 1;
  const bool big = streams(IN, p.rows, p.N, p.K, p.groups);
  if (p.rows <= kRowsMax) return run_rows<IN, EP>(out_type, p, big, st);
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
  const long want = ((long)p.rows * ceil_div(p.N / G, 256) + 3) / 4;
  const unsigned blocks = (unsigned)(want < 4096 ? want : 4096);
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
