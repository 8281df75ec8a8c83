// csrc/gelu_tail.hpp for the host: the polynomial in f32, as the kernels evaluate it, and
// in f64 with the same coefficients.
#include <math.h>

#include "../../moe_expert_layer_sigmoid_amd/csrc/gelu_tail.hpp"

extern "C" float gelu_tail_f32(float a) {
  const float t = 1.0f / fmaf(moe::kTailArg, a, 1.0f);
  float q = moe::kTail[moe::kTailDegree];
  for (int i = moe::kTailDegree - 1; i >= 0; --i) q = fmaf(q, t, moe::kTail[i]);
  return t * q;
}

extern "C" double gelu_tail_f64(double a) {
  const double t = 1.0 / (moe::kTailArg * a + 1.0);
  double q = moe::kTail[moe::kTailDegree];
  for (int i = moe::kTailDegree - 1; i >= 0; --i) q = q * t + moe::kTail[i];
  return t * q;
}
