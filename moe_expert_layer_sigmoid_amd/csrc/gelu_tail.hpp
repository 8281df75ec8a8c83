// The normal distribution's scaled tail, Phi(-a) e^(a^2 / 2), as a polynomial (host
// and device).
#pragma once

namespace moe {

// For a >= 0 it is t Q(t) with t = 1 / (1 + kTailArg a).  Q was fitted to the scaled
// complementary error function for the least largest relative error over 0 <= a <= 27, with
// Q(1) = 0.5, the value at a = 0, which most activations are near; then each coefficient
// was rounded to f32 and the others fitted again.  5.2e-8 as they stand, 6 x 2^-24
// with f32's roundings.
constexpr float kTailArg = 0.27f;
constexpr int kTailDegree = 8;
constexpr float kTail[kTailDegree + 1] = {0.107719138f,   0.107579179f, 0.101473309f,  0.0736839175f, 0.103239618f,
                                          -0.0614932701f, 0.162113652f, -0.122336753f, 0.0280212089f};

}  // namespace moe
