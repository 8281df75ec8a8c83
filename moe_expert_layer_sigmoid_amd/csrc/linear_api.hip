// C ABI of the linear operators: host-side validation in front of their
// launches (see include/moe.h for the contract).

#include <hip/hip_runtime.h>

#include "../../include/moe.h"
#include "linear_internal.hpp"

using namespace moe;

namespace {

static_assert((int)kBF16 == MOE_TYPE_BF16 && (int)kF16 == MOE_TYPE_F16 && (int)kF32 == MOE_TYPE_F32 &&
                  (int)kFP8 == MOE_TYPE_FP8,
              "type codes");

constexpr int kMaxWidth = 32768;
constexpr int kMaxGroups = 1024;
constexpr int kMaxRows = 1 << 20;

bool aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool dev_ok(const void* p) { return p != nullptr && aligned(p); }
bool opt_ok(const void* p) { return aligned(p); }
// a tensor of `rows` rows: it may be missing when there are none
bool rows_ok(const void* p, int rows) { return rows == 0 ? opt_ok(p) : dev_ok(p); }
int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

int check_linear(const moe_linear_t* d) {
  if (!d || d->rows < 0 || d->N < 1 || d->K < 1 || d->groups < 1) return MOE_ERR_INVALID_ARG;
  if (d->rows > kMaxRows || d->N > kMaxWidth || d->K > kMaxWidth || d->groups > kMaxGroups) return MOE_ERR_UNSUPPORTED;
  if (d->in_type == MOE_TYPE_FP8) {
    if (d->out_type < MOE_TYPE_BF16 || d->out_type > MOE_TYPE_F32) return MOE_ERR_INVALID_ARG;
    return d->K % 16 ? MOE_ERR_INVALID_ARG : MOE_OK;
  }
  if (d->in_type != MOE_TYPE_BF16 && d->in_type != MOE_TYPE_F16) return MOE_ERR_INVALID_ARG;
  if (d->out_type != d->in_type && d->out_type != MOE_TYPE_F32) return MOE_ERR_INVALID_ARG;
  return d->K % 8 ? MOE_ERR_INVALID_ARG : MOE_OK;
}

int check_call(const moe_linear_t* d, const int32_t* offsets, const void* ws, size_t bytes) {
  if (!offsets && d->groups != 1) return MOE_ERR_INVALID_ARG;
  if (!opt_ok(offsets)) return MOE_ERR_INVALID_ARG;
  const size_t need = linear_workspace(d->rows, d->N, d->K, d->groups, d->in_type);
  if (need && (!ws || bytes < need)) return MOE_ERR_WORKSPACE;
  return opt_ok(ws) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

int quant(bool swiglu, int32_t rows, int32_t K, int32_t x_type, const void* x, int64_t ldx, uint8_t* q, float* qs,
          moe_stream_t stream) {
  if (rows < 0 || K < 1 || K % 16 || x_type < MOE_TYPE_BF16 || x_type > MOE_TYPE_F32) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRows || K > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  if (ldx % 16 || ldx < (int64_t)K * (swiglu ? 2 : 1)) return MOE_ERR_INVALID_ARG;
  if (ldx > ((int64_t)1 << 40)) return MOE_ERR_UNSUPPORTED;
  if (!rows_ok(x, rows) || !rows_ok(q, rows) || !rows_ok(qs, rows)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  return hip_status(launch_fp8_quant(x, x_type, swiglu, rows, K, ldx, q, qs, (hipStream_t)stream));
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_bytes(const moe_linear_t* d) {
  return check_linear(d) == MOE_OK ? linear_workspace(d->rows, d->N, d->K, d->groups, d->in_type) : 0;
}

int moe_fp8_quant(int32_t rows, int32_t K, int32_t x_type, const void* x, int64_t ldx, uint8_t* q, float* qs,
                  moe_stream_t stream) {
  return quant(false, rows, K, x_type, x, ldx, q, qs, stream);
}

int moe_fp8_swiglu_quant(int32_t rows, int32_t K, int32_t x_type, const void* x, int64_t ldx, uint8_t* q, float* qs,
                         moe_stream_t stream) {
  return quant(true, rows, K, x_type, x, ldx, q, qs, stream);
}

int moe_fp8_linear(const moe_linear_t* d, const uint8_t* xq, const float* xs, const uint8_t* w, const float* ws,
                   const int32_t* offsets, void* y, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_linear(d);
  if (rc) return rc;
  if (d->in_type != MOE_TYPE_FP8 || !rows_ok(xq, d->rows) || !rows_ok(xs, d->rows) || !dev_ok(w) || !dev_ok(ws) ||
      !rows_ok(y, d->rows))
    return MOE_ERR_INVALID_ARG;
  if ((rc = check_call(d, offsets, workspace, workspace_bytes))) return rc;
  if (d->rows == 0) return MOE_OK;
  const LinearArgs p{w, xq, ws, xs, offsets, y, d->rows, d->N, d->K, d->groups, nullptr};
  return hip_status(launch_linear(kFwd, d->in_type, d->out_type, p, workspace, (hipStream_t)stream));
}

int moe_grouped_linear(const moe_linear_t* d, const void* x, const void* w, const int32_t* offsets, void* y,
                       void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_linear(d);
  if (rc) return rc;
  if (d->in_type == MOE_TYPE_FP8 || !rows_ok(x, d->rows) || !dev_ok(w) || !rows_ok(y, d->rows))
    return MOE_ERR_INVALID_ARG;
  if ((rc = check_call(d, offsets, workspace, workspace_bytes))) return rc;
  if (d->rows == 0) return MOE_OK;
  const LinearArgs p{w, x, nullptr, nullptr, offsets, y, d->rows, d->N, d->K, d->groups, nullptr};
  return hip_status(launch_linear(kFwd, d->in_type, d->out_type, p, workspace, (hipStream_t)stream));
}

int moe_grouped_linear_dx(const moe_linear_t* d, const void* dy, const void* w, const int32_t* offsets, void* dx,
                          void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_linear(d);
  if (rc) return rc;
  if (d->in_type == MOE_TYPE_FP8 || d->N % 8 || !rows_ok(dy, d->rows) || !dev_ok(w) || !rows_ok(dx, d->rows))
    return MOE_ERR_INVALID_ARG;
  if ((rc = check_call(d, offsets, workspace, workspace_bytes))) return rc;
  if (d->rows == 0) return MOE_OK;
  const LinearArgs p{w, dy, nullptr, nullptr, offsets, dx, d->rows, d->N, d->K, d->groups, nullptr};
  return hip_status(launch_linear(kDx, d->in_type, d->out_type, p, workspace, (hipStream_t)stream));
}

int moe_grouped_linear_dw(const moe_linear_t* d, const void* dy, const void* x, const int32_t* offsets, void* dw,
                          void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_linear(d);
  if (rc) return rc;
  if (d->in_type == MOE_TYPE_FP8 || d->N % 8 || !rows_ok(dy, d->rows) || !rows_ok(x, d->rows) || !dev_ok(dw))
    return MOE_ERR_INVALID_ARG;
  if ((rc = check_call(d, offsets, workspace, workspace_bytes))) return rc;
  const LinearArgs p{x, dy, nullptr, nullptr, offsets, dw, d->rows, d->N, d->K, d->groups, nullptr};
  return hip_status(launch_linear(kDw, d->in_type, d->out_type, p, workspace, (hipStream_t)stream));
}

}  // extern "C"
