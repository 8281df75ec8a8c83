// The gradient through bias and activation of a product by expert: from dy =
// dL/dy and z (the values before the activation),
//   dz = dy act'(z),  or with z = (gate, up):  dz = (dy up act'(gate), dy act(gate)),
//   db_g = sum over the group's rows of dz (f32, before dz is rounded).
// One pass, bound by memory: 49152 rows of 48 groups, 4096 columns gated, 213 us for
// 1.0 GB (4.7 TB/s; a copy reaches 5.2) and 8 for the sums.  A block takes a tile of
// rows of one group and all columns that 256 threads hold, eight a thread, so that a
// column's sum stays in registers and crosses threads once, through LDS.  The tiles are
// as long as it takes for the card to hold all of them at a time: no second round of
// blocks that leaves most of it idle.  A tile's sums are f32 partial sums in the
// workspace, added in row order by a second launch.  Up to 256 rows in all, a block
// takes all rows of a group and few columns, and writes db itself (250 rows of 9 groups,
// 264 columns: 5.7 us, in two launches 8.5).

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_kernel.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kV = 8;           // columns a thread
constexpr int kWhole = 256;     // rows up to which a group's columns may be one block's
constexpr int kWholeRows = 8;   // ... and of a thread, one after the other
constexpr int kFewRows = 4;     // rows of a thread up to which it has two in flight
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
template <int IN, int PT, int EP, int ACT, int kAhead>
__global__ void __launch_bounds__(kThreads, resident(EP)) k_act_backward(ActBackwardArgs p, int per, int ncb, int len, bool once, float* sums) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int G = EP == kGated ? 2 : 1;
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
#pragma unroll 8
    for (int t = 1; t < subs; ++t) s += red[w + t * per][k];
    sums[(size_t)tile * p.N + k / kV * n_out + col] = s;
  }
#endif
}

// db[g] = the group's partial sums, the tiles dealt to the threads of a column in
// runs, the runs' sums added in pairs.  across: threads (of four columns) across a
// block: 16, or 4 where so few columns leave most of the card idle (38808 rows of
// 216: both launches 22.2 us, with 16 24.0).  tiles: that the workspace holds (offsets that fall, against the
// contract, would count more).
__global__ void __launch_bounds__(kThreads) k_act_backward_join(const float* part, const int32_t* off, int rows, int N, int len,
                                                                int tiles, int across, float* db) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ v4f red[kThreads / 64][16];
  const int g = blockIdx.y, lane = threadIdx.x & 63, slices = kThreads / across;
  const int col = threadIdx.x % across, slice = threadIdx.x / across;
  const int c = (blockIdx.x * across + col) * 4;  // N % 8 == 0
  int before = 0, lo, hi;                         // tiles of the groups before
  for (int k = lane; k < g; k += 64) {
    group_rows(off, k, rows, lo, hi);
    before += (hi - lo + len - 1) / len;
  }
#pragma unroll
  for (int d = 32; d; d /= 2) before += __shfl_xor(before, d);
  group_rows(off, g, rows, lo, hi);
  const int n = min((hi - lo + len - 1) / len, max(0, tiles - before)), each = (n + slices - 1) / slices;
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
  for (int d = across; d < 64; d *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += __shfl_xor(s[e], d);
  if (lane < across) red[threadIdx.x / 64][lane] = s;
  __syncthreads();
  if (slice == 0 && c < N) {
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) s += red[w][col];
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

// Threads across a block that takes all rows of a group: 8 (128 bytes of a row), fewer
// where a thread would have more than kWholeRows / 4 rows should one group hold
// them all, more where the blocks would be too many; 0 if kWholeRows are then not enough.
// What a thread has to compute counts here, with one wave a SIMD: gelu_tanh, 64 rows of
// 4096 columns, gated, 6.0 us, 69 by 256 threads across; 512 rows of 256 columns with 16
// rows a thread 20, with 4 9.3, in two launches 9.0.
int whole_across(int rows, int n_out, int groups) {
  const int chunks = ceil_div(n_out, kV);
  int per = 8;
  while (per > 2 && rows * per > kWholeRows / 4 * kThreads) per /= 2;
  while (per < kThreads && (long)groups * ceil_div(chunks, per) > 4 * kCus * resident(kAct)) per *= 2;
  if (per > chunks) per = chunks;
  return rows <= kWhole && rows * per <= kWholeRows * kThreads ? per : 0;
}

template <int IN, int PT, int EP>
hipError_t run(const ActBackwardArgs& p, void* ws, hipStream_t st) {
  const int n_out = p.N / (EP == kGated ? 2 : 1), across = p.db ? whole_across(p.rows, n_out, p.groups) : 0;
  const bool whole = across > 0;
  Division d = divide(p.rows, n_out, p.groups, EP);
  if (whole) {
    d.per = across;
    d.ncb = ceil_div(ceil_div(n_out, kV), across);
  }
  float* sums = whole ? p.db : p.db ? static_cast<float*>(ws) : nullptr;
  const unsigned blocks = (unsigned)((whole ? p.groups : d.tiles) * d.ncb);
  // what passes the caches moves with the streaming policy
  const bool once = (size_t)p.rows * p.N * 4 > kStreamMin;
  // (few rows a thread: the code of four side by side takes longer to load than it saves;
  // 256 rows of 48 groups, 4096 columns 9.4 us for 11.0)
  const bool few = whole || d.len * d.per <= kFewRows * kThreads;
  const auto launch = [&](auto a) {
    constexpr int ACT = decltype(a)::value, kMost = PT == kF32 ? 2 : 4;
    if (few) k_act_backward<IN, PT, EP, ACT, 2><<<blocks, kThreads, 0, st>>>(p, d.per, d.ncb, whole ? 0 : d.len, once, sums);
    else k_act_backward<IN, PT, EP, ACT, kMost><<<blocks, kThreads, 0, st>>>(p, d.per, d.ncb, d.len, once, sums);
  };
  with_act(p.act, launch);
  if (p.db && !whole) {
    const int wide = (long)ceil_div(p.N, 64) * p.groups < kCus ? 4 : 16;
    k_act_backward_join<<<dim3((unsigned)ceil_div(p.N, 4 * wide), p.groups), kThreads, 0, st>>>(sums, p.off, p.rows, p.N, d.len,
                                                                                                d.tiles, wide, p.db);
  }
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
  const int half = N / 2 > 0 ? N / 2 : 1;
  if (whole_across(rows, N, groups) && whole_across(rows, half, groups)) return 0;
  const int a = divide(rows, N, groups, kAct).tiles, b = divide(rows, half, groups, kGated).tiles;
  return (size_t)(a > b ? a : b) * N * sizeof(float);
}

}  // namespace moe
