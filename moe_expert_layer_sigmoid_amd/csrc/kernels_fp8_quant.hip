// fp8 quantisation with one f32 scale per row and 128 columns, plain and
// behind SwiGLU:
//   s = max(amax |v| / 448, 2^-126),  q = e4m3_rne(v * (1 / s)),
// v = x, or silu(gate) * up in f32.  The division, the reciprocal and the
// product are correctly rounded f32, so the codes of the plain form are those of
// the same formula evaluated anywhere in f32 (silu's exponential and reciprocal
// are the hardware's; see silu_mul).  The floor 2^-126 keeps 1 / s finite for
// blocks of zeros.  A block holding a NaN or an infinity gets a scale that is
// NaN or infinite, as the formula says (amax is taken with NaN kept).

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_internal.hpp"
#include "moe_device.hpp"

namespace moe {
namespace {

constexpr int kQuantThreads = 256;

constexpr int kPer = 16;  // columns per thread: one 16-byte store of codes

// kPer values at p (16-byte aligned) as f32
template <int XT>
__device__ __forceinline__ void load_row(const void* p, size_t i, float (&v)[kPer]) {
  if constexpr (XT == kF32) {
    const v4f* s = reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) {
      const v4f x = s[k];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * k + e] = x[e];
    }
  } else {
    typedef _Float16 v8h __attribute__((ext_vector_type(8)));
    const v4i* s = reinterpret_cast<const v4i*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int k = 0; k < kPer / 8; ++k) {
      const v4i x = s[k];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (XT == kBF16)
          v[8 * k + e] = __uint_as_float((e & 1) ? (uint32_t)x[e / 2] & 0xFFFF0000u : (uint32_t)x[e / 2] << 16);
        else
          v[8 * k + e] = (float)__builtin_bit_cast(v8h, x)[e];
      }
    }
  }
}

// e^-g from the hardware's exp2 (1 ulp), its argument carried in two parts:
// one f32 product -g log2(e) would lose log2|g| bits of the result.
__device__ __forceinline__ float exp_neg(float g) {
  const float hi = g * -1.44269504f;
  const float lo = fmaf(g, -1.44269504f, -hi) + g * -1.92596299e-8f;  // log2(e) = 1.44269504 + 1.92596299e-8
  return __builtin_amdgcn_exp2f(hi) * fmaf(lo, 0.69314718f, 1.0f);
}

// silu(g) u for g >= kFarGate: the hardware's reciprocal (1 ulp) in place of a
// division keeps the kernel on the memory's side of its balance (in all within
// 9 x 2^-24 of the value, far below the codes' 2^-4).  Above 88 the sigmoid
// rounds to 1, and e^-inf by the two parts above would be NaN.
constexpr float kFarGate = -80.0f;
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float e = exp_neg(g);
  const float r = g > 88.0f ? 1.0f : __builtin_amdgcn_rcpf(1.0f + e);
  return g * r * u;
}

// silu(g) u for g < kFarGate, where 1 + e^-g rounds to e^-g: g e^g u.  Below
// -87 neither e^g nor its reciprocal is a normal f32, while the product may be
// one (silu(-88) = -5e-37, times u): t = e^(g/4) is normal down to -349, where
// no u brings the product back into range, and every partial product is
// normal wherever the result is (four errors of t and five roundings: 21 x
// 2^-24).  g = -inf: NaN, as in the formula.
__device__ __forceinline__ float silu_mul_far(float g, float u) {
  const float t = exp_neg(-0.25f * g);
  return (g * t) * (u * t) * t * t;
}

// One thread per 16 columns, 8 threads per block of 128: every load and store
// is 16 bytes.  Bound by memory: 14.9 us at 8192 x 2048 behind SwiGLU (84 MB, 5.6
// TB/s; a copy reaches 5.0); 8-column threads with scalar loads took 34.3.
template <int XT, bool SWIGLU>
__global__ void __launch_bounds__(kQuantThreads)
    k_fp8_quant(const void* __restrict__ x, int rows, int K, int64_t ldx, uint8_t* __restrict__ q,
                float* __restrict__ qs) {
  const uint32_t nb = (uint32_t)(K + 127) / 128;
  const uint32_t unit = (blockIdx.x * kQuantThreads + threadIdx.x) / 8;  // rows * nb <= 2^28
  if (unit >= (uint32_t)rows * nb) return;  // whole groups of 8 lanes
  const uint32_t row = unit / nb, b = unit - row * nb;
  const int c = (int)b * 128 + (threadIdx.x & 7) * kPer;
  float v[kPer] = {};
  if (c < K) {  // K % 16 == 0
    load_row<XT>(x, row * ldx + c, v);
    if constexpr (SWIGLU) {
      float u[kPer];
      load_row<XT>(x, row * ldx + K + c, u);
      float g[kPer];
      bool far = false;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        g[i] = v[i];
        far |= g[i] < kFarGate;
        v[i] = silu_mul(g[i], u[i]);
      }
      if (far) {  // one branch for all columns: no trained model's gates get there
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (g[i] < kFarGate) v[i] = silu_mul_far(g[i], u[i]);
      }
    }
  }
  // as bits: magnitudes order like integers, infinity above them, NaN above all
  uint32_t mb = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) mb = max(mb, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d < 8; d *= 2) mb = max(mb, (uint32_t)__shfl_xor((int)mb, d));
  const float s0 = __uint_as_float(mb) / 448.0f;
  const float s = s0 < 0x1p-126f ? 0x1p-126f : s0;
  const float inv = 1.0f / s;
  if (c < K) {
    v4i o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = (int)pack4_fp8(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    *reinterpret_cast<v4i*>(q + (size_t)row * K + c) = o;
  }
  if ((threadIdx.x & 7) == 0) qs[unit] = s;
}

template <int XT, bool SWIGLU>
hipError_t run_quant(const void* x, int rows, int K, int64_t ldx, uint8_t* q, float* qs, hipStream_t st) {
  const size_t threads = (size_t)rows * ((K + 127) / 128) * 8;
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
