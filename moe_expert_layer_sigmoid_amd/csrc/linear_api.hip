// C ABI of the linear operators: host-side validation in front of their
// launches (see include/moe.h for the contract).

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "../../include/moe.h"
#include "act_device.hpp"
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

int check_act(const moe_linear_t* d, int32_t act, int32_t gated) {
  const int rc = check_linear(d);
  if (rc) return rc;
  if (d->in_type == MOE_TYPE_FP8 || act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH || (gated != 0 && gated != 1) ||
      (gated && d->N % 2))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

size_t act_workspace(const moe_linear_t* d) {
  const size_t a = linear_workspace(d->rows, d->N, d->K, d->groups, d->in_type);
  const size_t b = act_backward_workspace(d->rows, d->N, d->groups);
  return a > b ? a : b;
}

int check_tensors(const moe_tensor_t* t, int32_t count, bool outs) {
  if (count < 0 || (count && !t)) return MOE_ERR_INVALID_ARG;
  if (count > MOE_GRAD_MAX_TENSORS) return MOE_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n < 0 || t[i].type < MOE_TYPE_BF16 || t[i].type > MOE_TYPE_F32) return MOE_ERR_INVALID_ARG;
    if (t[i].n > ((int64_t)1 << 36)) return MOE_ERR_UNSUPPORTED;
    const uintptr_t size = t[i].type == MOE_TYPE_F32 ? 4 : 2;
    if (t[i].n && (!t[i].in || (uintptr_t)t[i].in % size)) return MOE_ERR_INVALID_ARG;
    if (t[i].n && outs && (!t[i].out || (uintptr_t)t[i].out % size)) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

static_assert(sizeof(moe_tensor_t) == sizeof(GradTensor) && offsetof(moe_tensor_t, n) == offsetof(GradTensor, n) &&
                  offsetof(moe_tensor_t, type) == offsetof(GradTensor, type),
              "tensor lists are passed on as they are");
static_assert((int)kActNone == MOE_ACT_NONE && (int)kActRelu == MOE_ACT_RELU && (int)kActSilu == MOE_ACT_SILU &&
                  (int)kActGelu == MOE_ACT_GELU && (int)kActGeluTanh == MOE_ACT_GELU_TANH,
              "activation codes");

int check_grad(const moe_tensor_t* t, int32_t count, bool outs, void* ws, size_t bytes) {
  const int rc = check_tensors(t, count, outs);
  if (rc) return rc;
  if (!ws || bytes < grad_workspace(count)) return MOE_ERR_WORKSPACE;
  return aligned(ws) ? MOE_OK : MOE_ERR_INVALID_ARG;
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

size_t moe_linear_act_workspace_bytes(const moe_linear_t* d) {
  return check_act(d, MOE_ACT_NONE, 0) == MOE_OK ? act_workspace(d) : 0;
}

int moe_grouped_linear_act(const moe_linear_t* d, int32_t act, int32_t gated, const void* x, const void* w,
                           const void* bias, const void* residual, const int32_t* offsets, void* y, void* pre,
                           void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_act(d, act, gated);
  if (rc) return rc;
  if (!rows_ok(x, d->rows) || !dev_ok(w) || !rows_ok(y, d->rows) || !opt_ok(bias) || !opt_ok(residual) || !opt_ok(pre))
    return MOE_ERR_INVALID_ARG;
  if ((rc = check_call(d, offsets, workspace, workspace_bytes))) return rc;
  if (d->rows == 0) return MOE_OK;
  LinearArgs p{w, x, nullptr, nullptr, offsets, y, d->rows, d->N, d->K, d->groups, nullptr};
  p.bias = bias;
  p.res = residual;
  p.pre = pre;
  p.act = act;
  const auto launch = d->in_type == MOE_TYPE_BF16 ? launch_linear_act_bf16 : launch_linear_act_f16;
  return hip_status(launch(d->out_type, gated != 0, p, workspace, (hipStream_t)stream));
}

int moe_grouped_linear_act_backward(const moe_linear_t* d, int32_t act, int32_t gated, const void* dy, const void* pre,
                                    const int32_t* offsets, void* dz, float* db, void* workspace,
                                    size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_act(d, act, gated);
  if (rc) return rc;
  if (d->N % 8 || !rows_ok(dy, d->rows) || !rows_ok(pre, d->rows) || !rows_ok(dz, d->rows) || !opt_ok(db))
    return MOE_ERR_INVALID_ARG;
  if ((!offsets && d->groups != 1) || !opt_ok(offsets) || !opt_ok(workspace)) return MOE_ERR_INVALID_ARG;
  const size_t need = db ? act_backward_workspace(d->rows, d->N, d->groups) : 0;
  if (need && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
  if (d->rows == 0 && !db) return MOE_OK;
  const ActBackwardArgs p{dy, pre, offsets, dz, db, d->rows, d->N, d->groups, act};
  return hip_status(launch_act_backward(d->in_type, d->out_type, gated != 0, p, workspace, (hipStream_t)stream));
}

size_t moe_grad_workspace_bytes(int32_t count) {
  return count >= 0 && count <= MOE_GRAD_MAX_TENSORS ? grad_workspace(count) : 0;
}

int moe_grad_norm(const moe_tensor_t* tensors, int32_t count, float* norm, void* workspace, size_t workspace_bytes,
                  moe_stream_t stream) {
  const int rc = check_grad(tensors, count, false, workspace, workspace_bytes);
  if (rc) return rc;
  if (!norm || (uintptr_t)norm % 4) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_grad_norm(reinterpret_cast<const GradTensor*>(tensors), count, norm, workspace, (hipStream_t)stream));
}

int moe_grad_clip(const moe_tensor_t* tensors, int32_t count, float max_norm, float* norm, void* workspace,
                  size_t workspace_bytes, moe_stream_t stream) {
  const int rc = check_grad(tensors, count, true, workspace, workspace_bytes);
  if (rc) return rc;
  if (!(max_norm >= 0.0f) || (uintptr_t)norm % 4) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_grad_clip(reinterpret_cast<const GradTensor*>(tensors), count, max_norm, norm, workspace,
                                     (hipStream_t)stream));
}

}  // extern "C"
