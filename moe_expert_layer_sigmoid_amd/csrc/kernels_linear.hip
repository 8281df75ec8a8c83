// Linear operators on gfx950's matrix instructions: the fp8 product with a
// scale per block of 128, and the 16-bit products grouped by expert, forward
// and both gradients.
//
// One kernel template over the operand types and the three products.  The
// output's contiguous dimension ("columns") is the MFMA's A side, so that a
// lane holds four consecutive columns of one row; its rows are the B side.
//   y[row, n]   : A = w  [n][k],  B = x [row][k],   reduced over k
//   dx[row, k]  : A = w  [n][k]^T, B = dy [row][n], reduced over n
//   dw[n, k]    : A = x  [row][k]^T, B = dy [row][n]^T, reduced over rows
// An operand whose reduction is not contiguous is transposed on its way into
// LDS.  fp8: the four scales of a 128-column stage are constant over it, so
// one 16x16x128 product per tile is scaled by xs * ws in f32 and added to an
// f32 accumulator.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_internal.hpp"
#include "moe_device.hpp"

namespace moe {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kTile = 64;       // columns and rows of a block's output tile
constexpr int kPitch = 128 + 16;  // bytes of a staged row: 128 of data, padded against bank conflicts

template <int IN>
__device__ __forceinline__ v4f mfma16(v4i a, v4i b, v4f c) {  // 16x16x32, 16-bit types
  if constexpr (IN == kBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// 16x16x128 of e4m3 operands, no block scales
__device__ __forceinline__ v4f mfma8(v8i a, v8i b, v4f c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, kFmtFp8, kFmtFp8, 0, 0, 0, 0);
}

template <int OUT>
__device__ __forceinline__ void store1(void* out, size_t i, float v) {  // one rounding to the output type, to nearest even
  if constexpr (OUT == kBF16) static_cast<__bf16*>(out)[i] = (__bf16)v;
  else if constexpr (OUT == kF16) static_cast<_Float16*>(out)[i] = (_Float16)v;
  else static_cast<float*>(out)[i] = v;
}

// Rows [lo, hi) of group g.  Offsets outside [0, rows], or falling, break the
// caller's contract; they are clamped so that no row outside the tensors is
// touched.
__device__ __forceinline__ void group_rows(const int32_t* off, int g, int rows, int& lo, int& hi) {
  lo = off ? min(max(off[g], 0), rows) : 0;
  hi = off ? min(max(off[g + 1], lo), rows) : rows;
}

// The group that row tile `tile` (of TB rows, counted over the groups in
// order) belongs to and its index there; false past the last one.  Every wave
// does this by itself: 64 groups at a time, one per lane, prefix sums across
// the lanes.
template <int TB>
__device__ __forceinline__ bool find_tile(const int32_t* off, int groups, int rows, int tile, int& g, int& t) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int c = 0; c < groups; c += 64) {
    int lo = 0, hi = 0;
    if (c + lane < groups) group_rows(off, c + lane, rows, lo, hi);
    const int nt = (hi - lo + TB - 1) / TB;
    int incl = nt;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int up = __shfl_up(incl, d);
      if (lane >= d) incl += up;
    }
    const unsigned long long past = __ballot(base + incl > tile);
    if (past) {
      const int l = __ffsll(past) - 1;
      g = c + l;
      t = tile - base - __shfl(incl - nt, l);
      return true;
    }
    base += __shfl(incl, 63);
  }
  return false;
}

template <int IN, int OP, int OUT>
__global__ void __launch_bounds__(256) k_linear(LinearArgs p) {
  constexpr int ES = IN == kFP8 ? 1 : 2;
  constexpr int RE = 128 / ES;  // reduction elements per stage
  __shared__ __align__(16) uint8_t sa[kTile * kPitch], sb[kTile * kPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, q = lane >> 4;
  const int wa = wave & 1, wb = wave >> 1;
  const int cols = OP == kFwd ? p.N : p.K;
  const int c0 = blockIdx.x * kTile;

  // the tile's output rows and its reduction
  int g, r0, nr, nred;
  size_t out0;             // output index of the tile's (row 0, column 0)
  int lo, hi;
  if (OP == kDw) {
    g = blockIdx.z;
    group_rows(p.off, g, p.rows, lo, hi);
    r0 = blockIdx.y * kTile;
    nr = min(kTile, p.N - r0);
    nred = hi - lo;
    out0 = ((size_t)g * p.N + r0) * p.K + c0;
  } else {
    int t;
    if (!find_tile<kTile>(p.off, p.groups, p.rows, blockIdx.y, g, t)) return;  // whole block
    group_rows(p.off, g, p.rows, lo, hi);
    r0 = lo + t * kTile;
    nr = min(kTile, hi - r0);
    nred = OP == kFwd ? p.K : p.N;
    out0 = (size_t)r0 * cols + c0;
  }
  const uint8_t* wslab = static_cast<const uint8_t*>(p.a) + (OP == kDw ? 0 : (size_t)g * p.N * p.K * ES);

  // 16-byte piece `pc` of stage row `row` of an operand with a contiguous reduction
  auto stage_kc = [&](uint8_t* s, const uint8_t* src, int ld, int nrow, int e0) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int i = tid + 256 * m, row = i >> 3, pc = i & 7;
      const int e = e0 + pc * (16 / ES);
      v4i v = {0, 0, 0, 0};
      if (row < nrow && e < nred) v = *reinterpret_cast<const v4i*>(src + ((size_t)row * ld + e) * ES);
      *reinterpret_cast<v4i*>(s + row * kPitch + pc * 16) = v;
    }
  };
  // ... and of one whose columns are contiguous: 8 columns of reduction row `red`
  auto stage_mc = [&](uint8_t* s, const uint16_t* src, int ld, int ncol, int e0) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int i = tid + 256 * m, red = i >> 3, c = (i & 7) * 8;
      v4i v = {0, 0, 0, 0};
      if (c < ncol && e0 + red < nred) v = *reinterpret_cast<const v4i*>(src + (size_t)(e0 + red) * ld + c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint16_t*>(s + (c + j) * kPitch + 2 * red) = (uint16_t)((uint32_t)v[j >> 1] >> (16 * (j & 1)));
    }
  };

  v4f acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const int nkb = (p.K + 127) / 128, nnb = (p.N + 127) / 128;
  for (int e0 = 0; e0 < nred; e0 += RE) {
    if (OP == kFwd) {
      stage_kc(sa, wslab + (size_t)c0 * p.K * ES, p.K, p.N - c0, e0);
      stage_kc(sb, static_cast<const uint8_t*>(p.b) + (size_t)r0 * p.K * ES, p.K, nr, e0);
    } else if (OP == kDx) {
      stage_mc(sa, reinterpret_cast<const uint16_t*>(wslab) + c0, p.K, cols - c0, e0);
      stage_kc(sb, static_cast<const uint8_t*>(p.b) + (size_t)r0 * p.N * ES, p.N, nr, e0);
    } else {
      stage_mc(sa, static_cast<const uint16_t*>(p.a) + (size_t)lo * p.K + c0, p.K, cols - c0, e0);
      stage_mc(sb, static_cast<const uint16_t*>(p.b) + (size_t)lo * p.N + r0, p.N, nr, e0);
    }
    __syncthreads();
    v4i a[2][2], b[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[i][h] = *reinterpret_cast<const v4i*>(sa + (wa * 32 + i * 16 + l16) * kPitch + h * 64 + q * 16);
        b[i][h] = *reinterpret_cast<const v4i*>(sb + (wb * 32 + i * 16 + l16) * kPitch + h * 64 + q * 16);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float s = 0.0f;
      if constexpr (IN == kFP8) {
        const int row = wb * 32 + j * 16 + l16;
        const float xs = row < nr ? p.bs[(size_t)(r0 + row) * nkb + e0 / 128] : 0.0f;
        s = xs * p.as[((size_t)g * nnb + c0 / 128) * nkb + e0 / 128];  // the tile lies in one block of 128 columns
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (IN == kFP8) {
          v8i av, bv;
#pragma unroll
          for (int d = 0; d < 4; ++d) av[d] = a[i][0][d], av[4 + d] = a[i][1][d], bv[d] = b[j][0][d], bv[4 + d] = b[j][1][d];
          const v4f d = mfma8(av, bv, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[e], s, acc[i][j][e]);
        } else {
          acc[i][j] = mfma16<IN>(a[i][0], b[j][0], acc[i][j]);
          acc[i][j] = mfma16<IN>(a[i][1], b[j][1], acc[i][j]);
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = wa * 32 + i * 16 + 4 * q + e, r = wb * 32 + j * 16 + l16;
        if (r < nr && c0 + c < cols) store1<OUT>(p.out, out0 + (size_t)r * cols + c, acc[i][j][e]);
      }
}

template <int IN, int OP, int OUT>
hipError_t run_linear(const LinearArgs& p, hipStream_t st) {
  const unsigned ca = (unsigned)(((OP == kFwd ? p.N : p.K) + kTile - 1) / kTile);
  // row tiles: every group adds at most one partial tile
  const unsigned rb = OP == kDw ? (unsigned)((p.N + kTile - 1) / kTile)
                                : (unsigned)(p.rows / kTile + (p.rows < p.groups ? p.rows : p.groups));
  if (OP != kDw && rb == 0) return hipSuccess;
  k_linear<IN, OP, OUT><<<dim3(ca, rb, OP == kDw ? p.groups : 1), 256, 0, st>>>(p);
  return hipGetLastError();
}

template <int IN, int OP>
hipError_t run_out(int out_type, const LinearArgs& p, hipStream_t st) {
  if (out_type == kBF16) return run_linear<IN, OP, kBF16>(p, st);
  if (out_type == kF16) return run_linear<IN, OP, kF16>(p, st);
  return run_linear<IN, OP, kF32>(p, st);
}

template <int IN>
hipError_t run_op(int op, int out_type, const LinearArgs& p, hipStream_t st) {
  if (op == kFwd) return run_out<IN, kFwd>(out_type, p, st);
  if (op == kDx) return run_out<IN, kDx>(out_type, p, st);
  return run_out<IN, kDw>(out_type, p, st);
}

}  // namespace

size_t linear_workspace(int, int, int, int, int) { return 0; }

hipError_t launch_linear(int op, int in_type, int out_type, const LinearArgs& p, void*, hipStream_t st) {
  if (in_type == kFP8) return run_out<kFP8, kFwd>(out_type, p, st);
  return in_type == kBF16 ? run_op<kBF16>(op, out_type, p, st) : run_op<kF16>(op, out_type, p, st);
}

}  // namespace moe
