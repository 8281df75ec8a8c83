// What the linear operators choose for given sizes, for tests without a GPU.
#include "../../moe_expert_layer_sigmoid_amd/csrc/linear_plan.hpp"

// out: shape (-1: the kernel of few rows), columns and rows of its tile, splits,
// stages of a split (kDw: of equal groups), whether the weights stream
extern "C" void linear_plan(int op, int in_type, int rows, int N, int K, int groups, int* out) {
  using namespace moe;
  const Choice c = choose(op, in_type, rows, N, K, groups);
  out[0] = op == kFwd && few_rows(rows, N, groups) ? -1 : c.shape;
  out[1] = kCost[c.shape].ta;
  out[2] = kCost[c.shape].tb;
  out[3] = c.plan.splits;
  out[4] = c.plan.sps;
  out[5] = streams(in_type, rows, N, K, groups);
}
