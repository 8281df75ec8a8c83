// The gradient through bias and activation of a product by expert: from dy =
// dL/dy and z (the values before the activation),
//   dz = dy act'(z),  or with z = (gate, up):  dz = (dy up act'(gate), dy act(gate)),
//   db_g = sum over the group's rows of dz (f32, before dz is rounded).
// One pass, bound by memory: 49152 rows of 48 groups, 4096 columns gated, 213 us for
// 1.0 GB (4.7 TB/s; a copy reaches 5.2) and 8 for the sums.  A block takes a tile of rows of one group and all
// columns that 256 threads hold, eight a thread, so that a column's sum stays in
// registers and crosses threads once, through LDS.  The tiles are as long as it
// takes for the card to hold all of them at a time: no second round of blocks that
// leaves most of it idle.  A tile's sums are f32 partial sums in the workspace, added in
// row order by a second launch; up to kWhole rows in all a group is one block,
// which writes db itself.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_kernel.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kV = 8;        // columns a thread
constexpr int kWhole = 64;   // rows up to which a group is one block
// blocks that a compute unit's registers hold (gated: three operands in flight and twice the sums)
constexpr int resident(int ep) { return ep == kGated ? 3 : 4; }

template <int T>
using Elem = std::conditional_t<T == kBF16, __bf16, std::conditional_t<T == kF16, _Float16, float>>;

// Eight values as they lie in memory, zeros past the n that exist.
template <int T>
struct Raw {
  static constexpr int W = sizeof(Elem<T>) / 2;  // 16-byte words
  v4i w[W];
  __device__ __forceinline__ void load(const Elem<T>* p, int n, bool once) {
    if (n == kV) {
      const v4i_any* q = reinterpret_cast<const v4i_any*>(p);
#pragma unroll
      for (int h = 0; h < W; ++h) w[h] = once ? __builtin_nontemporal_load(q + h) : q[h];
    } else {
      Elem<T> x[kV];
#pragma unroll
      for (int e = 0; e < kV; ++e) x[e] = e < n ? p[e] : (Elem<T>)0.0f;
      __builtin_memcpy(w, x, sizeof(x));
    }
  }
  __device__ __forceinline__ void get(float (&v)[kV]) const {
    Elem<T> x[kV];
    __builtin_memcpy(x, w, sizeof(x));
#pragma unroll
    for (int e = 0; e < kV; ++e) v[e] = (float)x[e];
  }
};

template <int T>
__device__ __forceinline__ void store8(Elem<T>* p, int n, bool once, const float (&v)[kV]) {
  static_assert(T != kF32, "16 bytes");
  Elem<T> x[kV];
#pragma unroll
  for (int e = 0; e < kV; ++e) x[e] = (Elem<T>)v[e];
  if (n == kV) {
    v4i w;
    __builtin_memcpy(&w, x, 16);
    if (once) __builtin_nontemporal_store(w, reinterpret_cast<v4i_any*>(p));
    else store16(p, w);
  } else {
#pragma unroll
    for (int e = 0; e < kV; ++e)
      if (e < n) p[e] = x[e];
  }
}

// The group and rows of tile `tile` of `len` rows, counted over the groups in order
// (every wave by itself, 64 groups at a time); false if there are not so many.
__device__ __forceinline__ bool find_tile(const int32_t* off, int groups, int rows, int len, int tile, int& lo, int& hi) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int g = 0; g < groups; g += 64) {
    lo = hi = 0;
    if (g + lane < groups) group_rows(off, g + lane, rows, lo, hi);
    int n = (hi - lo + len - 1) / len;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int up = __shfl_up(n, d);
      if (lane >= d) n += up;
    }
    n += base;
    const unsigned long long past = __ballot(n > tile);
    if (past) {
      const int k = __ffsll(past) - 1;
      lo = __builtin_amdgcn_readlane(lo, k);
      hi = __builtin_amdgcn_readlane(hi, k);
      const int t = tile - (__builtin_amdgcn_readlane(n, k) - (hi - lo + len - 1) / len);
      lo += t * len;
      hi = min(hi, lo + len);
      return true;
    }
    base = __builtin_amdgcn_readlane(n, 63);
  }
  return false;
}

// per: threads across the columns of a block; ncb blocks across; len: rows of a
// tile, 0 for a group a block.  sums: the partial sums [tile][N], or db itself (len 0).
template <int IN, int PT, int EP, int ACT>
__global__ void __launch_bounds__(kThreads, resident(EP)) k_act_backward(ActBackwardArgs p, int per, int ncb, int len, bool once, float* sums) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int G = EP == kGated ? 2 : 1;
  constexpr int kAhead = PT == kF32 ? 2 : 4;  // rows a thread has in flight
  __shared__ float red[kThreads][G * kV + 1];
  const int n_out = p.N / G;
  const int tile = blockIdx.x / ncb, cb = blockIdx.x % ncb;
  int lo, hi;
  if (len == 0) group_rows(p.off, tile, p.rows, lo, hi);
  else if (!find_tile(p.off, p.groups, p.rows, len, tile, lo, hi)) return;
  const int sub = threadIdx.x / per, subs = kThreads / per;
  const int c = (cb * per + threadIdx.x % per) * kV;
  const int nc = sub < subs ? min(kV, n_out - c) : 0;
  const Elem<PT>* dy = static_cast<const Elem<PT>*>(p.dy) + c;
  const Elem<PT>* pre = static_cast<const Elem<PT>*>(p.pre) + c;
  Elem<IN>* dz = static_cast<Elem<IN>*>(p.dz) + c;

  float acc[G][kV] = {};
  if (nc > 0) {
    for (int r0 = lo + sub; r0 < hi; r0 += kAhead * subs) {
      Raw<PT> d[kAhead], z[kAhead][G];
#pragma unroll
      for (int m = 0; m < kAhead; ++m) {
        const size_t r = (size_t)min(r0 + m * subs, hi - 1);
        d[m].load(dy + r * n_out, nc, once);
#pragma unroll
        for (int h = 0; h < G; ++h) z[m][h].load(pre + r * p.N + h * n_out, nc, once);
      }
#pragma unroll
      for (int m = 0; m < kAhead; ++m) {
        const int r = r0 + m * subs;
        if (r >= hi) break;
        float v[kV], g[kV], u[kV], o[G][kV];
        d[m].get(v);
        z[m][0].get(g);
        z[m][G - 1].get(u);
        bool far = false;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
          float f, s;
          act_slope<ACT>(g[e], f, s);
          o[0][e] = (G == 2 ? v[e] * u[e] : v[e]) * s;
          if constexpr (G == 2) o[G - 1][e] = v[e] * f;
          far |= g[e] < far_below<ACT>();
        }
        if constexpr (ACT == kActSilu || ACT == kActGelu || ACT == kActGeluTanh) {
          if (far) {  // one branch for all columns: few or no values get there
#pragma unroll
            for (int e = 0; e < kV; ++e)
              if (g[e] < far_below<ACT>()) {
                float ignored;
                grad_far<ACT>(g[e], G == 2 ? v[e] * u[e] : v[e], v[e], o[0][e], G == 2 ? o[G - 1][e] : ignored);
              }
          }
        }
#pragma unroll
        for (int h = 0; h < G; ++h) {
#pragma unroll
          for (int e = 0; e < kV; ++e) acc[h][e] += o[h][e];
          store8<IN>(dz + (size_t)r * p.N + h * n_out, nc, once, o[h]);
        }
      }
    }
  }
  if (!sums) return;
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int e = 0; e < kV; ++e) red[threadIdx.x][h * kV + e] = acc[h][e];
  __syncthreads();
  // each sum by one thread, over the block's row classes in order
  for (int i = threadIdx.x; i < per * G * kV; i += kThreads) {
    const int w = i / (G * kV), k = i % (G * kV), col = (cb * per + w) * kV + k % kV;
    if (col >= n_out) continue;
    float s = red[w][k];
    for (int t = 1; t < subs; ++t) s += red[w + t * per][k];
    sums[(size_t)tile * p.N + k / kV * n_out + col] = s;
  }
#endif
}

// db[g] = the group's partial sums in order: 64 columns a block, four a thread, the
// tiles dealt to 16 threads a column in runs.  tiles: that the workspace holds
// (offsets that fall, against the contract, would count more).
__global__ void __launch_bounds__(256) k_act_backward_join(const float* part, const int32_t* off, int rows, int N, int len,
                                                           int tiles, float* db) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ v4f red[16][16];
  const int g = blockIdx.y, lane = threadIdx.x & 63, col = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int c = blockIdx.x * 64 + col * 4;  // N % 8 == 0
  int before = 0, lo, hi;                   // tiles of the groups before
  for (int k = lane; k < g; k += 64) {
    group_rows(off, k, rows, lo, hi);
    before += (hi - lo + len - 1) / len;
  }
#pragma unroll
  for (int d = 32; d; d /= 2) before += __shfl_xor(before, d);
  group_rows(off, g, rows, lo, hi);
  const int n = min((hi - lo + len - 1) / len, max(0, tiles - before)), each = (n + 15) / 16;
  const int t0 = min(n, slice * each), t1 = min(n, t0 + each);
  v4f s = {0.f, 0.f, 0.f, 0.f};
  if (c < N) {
    const float* p = part + (size_t)before * N + c;
    for (int t = t0; t < t1; t += 8) {
      v4f x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = *reinterpret_cast<const v4f*>(p + (size_t)min(t + k, t1 - 1) * N);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (t + k < t1) s += x[k];
    }
  }
  red[slice][col] = s;
  __syncthreads();
  if (slice == 0 && c < N) {
#pragma unroll
    for (int k = 1; k < 16; ++k) s += red[k][col];
    *reinterpret_cast<v4f*>(db + (size_t)g * N + c) = s;
  }
#endif
}

// How the rows are divided: threads across, blocks across, rows of a tile, tiles
// at most.  A tile has at least two rows a thread, and is so long that the tiles
// (a group's last one may be short) are no more than the card holds.
struct Division {
  int per, ncb, len, tiles;
};
Division divide(int rows, int n_out, int groups, int ep) {
  Division d;
  const int chunks = ceil_div(n_out, kV), live = rows < groups ? rows : groups;
  d.ncb = ceil_div(chunks, kThreads);
  d.per = ceil_div(chunks, d.ncb);
  const int least = 2 * (kThreads / d.per), most = ceil_div(kCus * resident(ep), d.ncb);
  const int want = ceil_div(rows, most - live > most / 2 ? most - live : ceil_div(most, 2));
  d.len = want > least ? want : least;
  d.tiles = rows / d.len + live;
  return d;
}

template <int IN, int PT, int EP>
hipError_t run(const ActBackwardArgs& p, void* ws, hipStream_t st) {
  const Division d = divide(p.rows, p.N / (EP == kGated ? 2 : 1), p.groups, EP);
  const bool whole = p.db && p.rows <= kWhole;
  float* sums = whole ? p.db : p.db ? static_cast<float*>(ws) : nullptr;
  const unsigned blocks = (unsigned)((whole ? p.groups : d.tiles) * d.ncb);
  // what passes the caches moves with the streaming policy
  const bool once = (size_t)p.rows * p.N * 4 > kStreamMin;
  const auto launch = [&](auto a) {
    k_act_backward<IN, PT, EP, decltype(a)::value><<<blocks, kThreads, 0, st>>>(p, d.per, d.ncb, whole ? 0 : d.len, once, sums);
  };
  with_act(p.act, launch);
  if (p.db && !whole)
    k_act_backward_join<<<dim3((unsigned)ceil_div(p.N, 64), p.groups), 256, 0, st>>>(sums, p.off, p.rows, p.N, d.len, d.tiles, p.db);
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

// (gated or not)
size_t act_backward_workspace(int rows, int N, int groups) {
  if (rows <= kWhole) return 0;
  const int a = divide(rows, N, groups, kAct).tiles, b = divide(rows, N / 2 > 0 ? N / 2 : 1, groups, kGated).tiles;
  return (size_t)(a > b ? a : b) * N * sizeof(float);
}

}  // namespace moe
