// The gradient through bias and activation of a product by expert: from dy =
// dL/dy and z (the values before the activation),
//   dz = dy act'(z),  or with z = (gate, up):  dz = (dy up act'(gate), dy act(gate)),
//   db_g = sum over the group's rows of dz (f32, before dz is rounded).
// One pass: a block takes up to kRows rows of one group and all columns that 256
// threads hold, eight a thread, so that a column's sum stays in a register and
// crosses threads once, through LDS.  A block's sums are f32 partial sums in the
// workspace, added in row order by a second launch; up to kRows rows in all a
// group is one block, which writes db itself.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_kernel.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = kActBackwardRows;
constexpr int kV = 8;        // columns a thread
constexpr int kAhead = 4;    // rows a thread has in flight

template <int T>
using Elem = std::conditional_t<T == kBF16, __bf16, std::conditional_t<T == kF16, _Float16, float>>;

// n <= 8 values at p as f32, zeros past them
template <int T>
__device__ __forceinline__ void load8(const Elem<T>* p, int n, float (&v)[kV]) {
  if (n == kV) {
    Elem<T> x[kV];
#pragma unroll
    for (int h = 0; h < (int)sizeof(x) / 16; ++h) {
      const v4i w = load16(reinterpret_cast<const char*>(p) + 16 * h);
      __builtin_memcpy(reinterpret_cast<char*>(x) + 16 * h, &w, 16);
    }
#pragma unroll
    for (int e = 0; e < kV; ++e) v[e] = (float)x[e];
  } else {
#pragma unroll
    for (int e = 0; e < kV; ++e) v[e] = e < n ? (float)p[e] : 0.0f;
  }
}

template <int T>
__device__ __forceinline__ void store8(Elem<T>* p, int n, const float (&v)[kV]) {
  static_assert(T != kF32, "16 bytes");
  Elem<T> x[kV];
#pragma unroll
  for (int e = 0; e < kV; ++e) x[e] = (Elem<T>)v[e];
  if (n == kV) {
    v4i w;
    __builtin_memcpy(&w, x, 16);
    store16(p, w);
  } else {
#pragma unroll
    for (int e = 0; e < kV; ++e)
      if (e < n) p[e] = x[e];
  }
}

// per: threads across the columns of a block; ncb blocks across.  sums: the
// partial sums [row tile][N], or db itself when `whole` (one block a group).
template <int IN, int PT, int EP>
__global__ void __launch_bounds__(kThreads) k_act_backward(ActBackwardArgs p, int per, int ncb, float* sums, bool whole) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int G = EP == kGated ? 2 : 1;
  __shared__ float red[kThreads][G * kV + 1];
  const int n_out = p.N / G;
  const int tile = blockIdx.x / ncb, cb = blockIdx.x % ncb;
  int lo, hi;
  if (whole) {
    group_rows(p.off, tile, p.rows, lo, hi);
  } else {
    const RowTiles<kRows> rt(p.off, p.groups, p.rows);
    if (tile >= rt.total) return;
    int g, t;
    rt.find(tile, g, t, lo, hi);
    lo += t * kRows;
    hi = min(hi, lo + kRows);
  }
  const int sub = threadIdx.x / per, subs = kThreads / per;
  const int c = (cb * per + threadIdx.x % per) * kV;
  const int nc = sub < subs ? min(kV, n_out - c) : 0;
  float acc[G][kV] = {};
  if (nc > 0) {
    const Elem<PT>* dy = static_cast<const Elem<PT>*>(p.dy) + c;
    const Elem<PT>* pre = static_cast<const Elem<PT>*>(p.pre) + c;
    Elem<IN>* dz = static_cast<Elem<IN>*>(p.dz) + c;
    with_act(p.act, [&](auto a) {
      constexpr int A = decltype(a)::value;
      for (int r0 = lo + sub; r0 < hi; r0 += kAhead * subs) {
        float d[kAhead][kV], z[kAhead][G][kV];
#pragma unroll
        for (int m = 0; m < kAhead; ++m) {
          const size_t r = (size_t)min(r0 + m * subs, hi - 1);
          load8<PT>(dy + r * n_out, nc, d[m]);
#pragma unroll
          for (int h = 0; h < G; ++h) load8<PT>(pre + r * p.N + h * n_out, nc, z[m][h]);
        }
#pragma unroll
        for (int m = 0; m < kAhead; ++m) {
          const int r = r0 + m * subs;
          if (r >= hi) break;
          float o[G][kV];
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            if constexpr (G == 2) {
              o[0][e] = slope_mul<A>(z[m][0][e], d[m][e] * z[m][G - 1][e]);
              o[G - 1][e] = act_mul<A>(z[m][0][e], d[m][e]);
            } else {
              o[0][e] = slope_mul<A>(z[m][0][e], d[m][e]);
            }
#pragma unroll
            for (int h = 0; h < G; ++h) acc[h][e] += o[h][e];
          }
#pragma unroll
          for (int h = 0; h < G; ++h) store8<IN>(dz + (size_t)r * p.N + h * n_out, nc, o[h]);
        }
      }
    });
  }
  if (!sums) return;
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int e = 0; e < kV; ++e) red[threadIdx.x][h * kV + e] = acc[h][e];
  __syncthreads();
  // each sum by one thread, over the block's row classes in order
  const int n = per * G * kV;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int w = i / (G * kV), k = i % (G * kV), col = (cb * per + w) * kV + k % kV;
    if (col >= n_out) continue;
    float s = red[w][k];
    for (int t = 1; t < subs; ++t) s += red[w + t * per][k];
    sums[(size_t)tile * p.N + k / kV * n_out + col] = s;
  }
#endif
}

// db[g] = the group's partial sums in order: 64 columns a block, the tiles dealt
// to 16 threads a column in runs.  tiles: that the workspace holds (offsets that
// fall, against the contract, would count more).
__global__ void __launch_bounds__(1024) k_act_backward_join(const float* part, const int32_t* off, int rows, int N,
                                                            int tiles, float* db) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ float red[16][64];
  const int g = blockIdx.y, lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  int before = 0, lo, hi;  // row tiles of the groups before
  for (int k = lane; k < g; k += 64) {
    group_rows(off, k, rows, lo, hi);
    before += (hi - lo + kRows - 1) / kRows;
  }
#pragma unroll
  for (int d = 32; d; d /= 2) before += __shfl_xor(before, d);
  group_rows(off, g, rows, lo, hi);
  const int n = min((hi - lo + kRows - 1) / kRows, max(0, tiles - before)), run = (n + 15) / 16;
  const int t0 = min(n, slice * run), t1 = min(n, t0 + run);
  float s = 0.0f;
  if (c < N) {
    const float* p = part + (size_t)before * N + c;
    for (int t = t0; t < t1; t += 8) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = p[(size_t)min(t + k, t1 - 1) * N];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (t + k < t1) s += x[k];
    }
  }
  red[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < N) {
#pragma unroll
    for (int k = 1; k < 16; ++k) s += red[k][lane];
    db[(size_t)g * N + c] = s;
  }
#endif
}

template <int IN, int PT, int EP>
hipError_t run(const ActBackwardArgs& p, void* ws, hipStream_t st) {
  const int chunks = ceil_div(p.N / (EP == kGated ? 2 : 1), kV);
  const int ncb = ceil_div(chunks, kThreads), per = ceil_div(chunks, ncb);
  const bool whole = p.db && p.rows <= kRows;
  const int live = p.rows < p.groups ? p.rows : p.groups;
  const unsigned tiles = (unsigned)(whole ? p.groups : p.rows / kRows + live);
  float* sums = whole ? p.db : p.db ? static_cast<float*>(ws) : nullptr;
  if (tiles) k_act_backward<IN, PT, EP><<<tiles * (unsigned)ncb, kThreads, 0, st>>>(p, per, ncb, sums, whole);
  if (p.db && !whole)
    k_act_backward_join<<<dim3((unsigned)ceil_div(p.N, 64), p.groups), 1024, 0, st>>>(sums, p.off, p.rows, p.N,
                                                                                              (int)tiles, p.db);
  return hipGetLastError();
}

template <int IN, int PT>
hipError_t run_gated(bool gated, const ActBackwardArgs& p, void* ws, hipStream_t st) {
  return gated ? run<IN, PT, kGated>(p, ws, st) : run<IN, PT, kAct>(p, ws, st);
}

}  // namespace

hipError_t launch_act_backward(int in_type, int out_type, bool gated, const ActBackwardArgs& p, void* ws, hipStream_t st) {
  if (in_type == kBF16)
    return out_type == kF32 ? run_gated<kBF16, kF32>(gated, p, ws, st) : run_gated<kBF16, kBF16>(gated, p, ws, st);
  return out_type == kF32 ? run_gated<kF16, kF32>(gated, p, ws, st) : run_gated<kF16, kF16>(gated, p, ws, st);
}

size_t act_backward_workspace(int rows, int N, int groups) {
  if (rows <= kRows) return 0;
  return ((size_t)(rows / kRows) + (size_t)(rows < groups ? rows : groups)) * N * sizeof(float);
}

}  // namespace moe
