// Products by expert with bias, activation and residual in the epilogue:
//   z = x w_g^T + b_g;   y = act(z) + r,  or  y = act(z[:, :F]) z[:, F:] + r  with N = 2 F.
// The kernels are the plain product's (linear_kernel.hpp), bound as it is; the
// epilogue works on sums that are in LDS for the turned stores anyway, so that z
// is never read back and each output is rounded once.

#include <hip/hip_runtime.h>

#include "linear_act_run.hpp"

namespace moe {

hipError_t launch_linear_act_bf16(int out_type, bool gated, const LinearArgs& p, void* ws, hipStream_t st) {
  return run_act<kBF16>(out_type, gated, p, ws, st);
}

}  // namespace moe
