// fp8 quantisation with one f32 scale per row and 128 columns, plain and
// behind SwiGLU:
//   s = max(amax |v| / 448, 2^-126),  q = e4m3_rne(v * (1 / s)),
// v = x, or silu(gate) * up in f32.  The division, the reciprocal and the
// product are correctly rounded f32, so the codes are those of the same
// formula evaluated anywhere in f32.  The floor 2^-126 keeps 1 / s finite for
// blocks of zeros.  A block holding a NaN or an infinity gets a scale that is
// NaN or infinite, as the formula says (amax is taken with NaN kept).

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_internal.hpp"
#include "moe_device.hpp"

namespace moe {
namespace {

constexpr int kQuantThreads = 256;

template <int XT>
__device__ __forceinline__ float to_f32(const void* p, size_t i) {
  if constexpr (XT == kBF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else if constexpr (XT == kF16) return (float)static_cast<const _Float16*>(p)[i];
  else return static_cast<const float*>(p)[i];
}

// larger of two magnitudes, NaN if either is
__device__ __forceinline__ float nan_max(float a, float b) { return (a > b || a != a) ? a : b; }

// One thread per 8 columns, 16 threads per block of 128.
template <int XT, bool SWIGLU>
__global__ void __launch_bounds__(kQuantThreads)
    k_fp8_quant(const void* __restrict__ x, int rows, int K, int64_t ldx, uint8_t* __restrict__ q,
                float* __restrict__ qs) {
  const int nb = (K + 127) / 128;
  const size_t unit = ((size_t)blockIdx.x * kQuantThreads + threadIdx.x) / 16;
  if (unit >= (size_t)rows * nb) return;  // whole groups of 16 lanes
  const size_t row = unit / nb;
  const int b = (int)(unit - row * nb);
  const int c = b * 128 + (threadIdx.x & 15) * 8;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.0f;
    if (c < K) {  // K % 8 == 0
      v[i] = to_f32<XT>(x, row * ldx + c + i);
      if (SWIGLU) v[i] = v[i] / (1.0f + expf(-v[i])) * to_f32<XT>(x, row * ldx + K + c + i);
    }
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = nan_max(fabsf(v[i]), m);
#pragma unroll
  for (int d = 1; d < 16; d *= 2) m = nan_max(m, __shfl_xor(m, d));
  const float s0 = m / 448.0f;
  const float s = s0 < 0x1p-126f ? 0x1p-126f : s0;
  const float inv = 1.0f / s;
  if (c < K) {
    v2i o;
    o.x = (int)pack4_fp8(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    o.y = (int)pack4_fp8(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    *reinterpret_cast<v2i*>(q + row * K + c) = o;
  }
  if ((threadIdx.x & 15) == 0) qs[unit] = s;
}

template <int XT, bool SWIGLU>
hipError_t run_quant(const void* x, int rows, int K, int64_t ldx, uint8_t* q, float* qs, hipStream_t st) {
  const size_t threads = (size_t)rows * ((K + 127) / 128) * 16;
  k_fp8_quant<XT, SWIGLU><<<(unsigned)((threads + kQuantThreads - 1) / kQuantThreads), kQuantThreads, 0, st>>>(
      x, rows, K, ldx, q, qs);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quant(const void* x, int x_type, bool swiglu, int rows, int K, int64_t ldx, uint8_t* q,
                            float* qs, hipStream_t st) {
  if (x_type == kBF16)
    return swiglu ? run_quant<kBF16, true>(x, rows, K, ldx, q, qs, st) : run_quant<kBF16, false>(x, rows, K, ldx, q, qs, st);
  if (x_type == kF16)
    return swiglu ? run_quant<kF16, true>(x, rows, K, ldx, q, qs, st) : run_quant<kF16, false>(x, rows, K, ldx, q, qs, st);
  return swiglu ? run_quant<kF32, true>(x, rows, K, ldx, q, qs, st) : run_quant<kF32, false>(x, rows, K, ldx, q, qs, st);
}

}  // namespace moe
