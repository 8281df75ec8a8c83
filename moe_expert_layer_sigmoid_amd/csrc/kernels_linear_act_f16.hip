// kernels_linear_act.hip's products on f16 operands.

#include <hip/hip_runtime.h>

#include "linear_act_run.hpp"

namespace moe {

hipError_t launch_linear_act_f16(int out_type, bool gated, const LinearArgs& p, void* ws, hipStream_t st) {
  return run_act<kF16>(out_type, gated, p, ws, st);
}

}  // namespace moe
