// The global norm over many tensors, sqrt(sum of squares), and the tensors
// scaled by min(1, max_norm / (norm + 1e-6)).
//
// Tensors are cut into chunks of kChunkElems values; a launch holds up to
// kTable tensors in its arguments (no table in memory that could go stale), and
// its blocks take equal runs of chunks.  A block's sum of squares is one f64
// partial sum: squares of f32 values keep their range and the sum all the bits
// that the result can show, whatever the order, and the order is fixed.  Every
// block of the scaling launch adds the partial sums (a few KB, from L2) itself
// and walks its run backwards, so that what the first pass read last is read first.
// Bound by memory: 528 M values in f32 342 us (6.2 TB/s) and 749 (5.6 TB/s, reads and
// writes; a copy reaches 5.2).

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_internal.hpp"
#include "moe_device.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 2048;        // partial sums of all launches together, and one a launch more
constexpr int kChunkElems = 16384;  // (8192: 1136 us for 1101 at 528 M values in f32)
constexpr int kTable = 168;          // with the rest 4072 bytes of arguments, under the 4 KB limit

struct Table {
  const void* in[kTable];
  void* out[kTable];
  uint32_t end[kTable];   // chunks up to the tensor's end
  uint32_t last[kTable];  // values of its last chunk, and above 16 bits its type
  int count;
  int part0;              // the launch's first partial sum
  uint32_t each, more;    // chunks of a block; the first `more` blocks take one more
};
static_assert(sizeof(Table) + 24 <= 4096 && kChunkElems < 1 << 16, "arguments");

typedef v4i v4i_any __attribute__((aligned(2)));

template <int T>
using Elem = std::conditional_t<T == kBF16, __bf16, std::conditional_t<T == kF16, _Float16, float>>;

// A block's run of chunks, and the tensor of its first (back: of its last): found by
// every wave with three loads at a time and ballots (36 tensors: 4.2 and 5.2 us a
// launch; by a binary search in the arguments, seven trips, 4.6 and 5.7).
struct Run {
  uint32_t c0, c1;
  int i;
  __device__ __forceinline__ Run(const Table& t, bool back) {
    const uint32_t b = blockIdx.x;
    c0 = b * t.each + min(b, t.more);
    c1 = c0 + t.each + (b < t.more ? 1 : 0);
    const uint32_t c = back ? c1 - 1 : c0;
    const int lane = threadIdx.x & 63;
    i = 0;  // tensors that end at or before c
#pragma unroll
    for (int k = 0; k < (kTable + 63) / 64; ++k) {
      const int j = 64 * k + lane;
      i += __popcll(__ballot(j < t.count && t.end[min(j, kTable - 1)] <= c));
    }
  }
};

// Calls f(tensor, first element, elements, type) for the run's chunks, in order or
// backwards.
template <class F>
__device__ __forceinline__ void chunks(const Table& t, const Run& run, bool back, F f) {
  int lo = run.i;
  for (uint32_t k = 0; k < run.c1 - run.c0; ++k) {
    const uint32_t c = back ? run.c1 - 1 - k : run.c0 + k;
    while (t.end[lo] <= c) ++lo;
    while (lo > 0 && t.end[lo - 1] > c) --lo;
    const uint32_t last = t.last[lo];
    const int64_t e0 = (int64_t)(c - (lo ? t.end[lo - 1] : 0)) * kChunkElems;
    f(lo, e0, c + 1 == t.end[lo] ? (int)(last & 0xFFFF) : kChunkElems, (int)(last >> 16));
  }
}

// One chunk, 16 bytes a thread and step: f(values, count, index of the first) for
// full and partial pieces.  LAST: the values are not needed again.  (Loads and
// stores of the scaling pass with the streaming policy, the first pass with the default one,
// leave the most in the memory-side cache: 528 M values in f32 1137 us, 1214 with
// the default everywhere, 1163 with streaming loads in the first pass alone; 44 M 86, 115, 110.)
template <int T, bool LAST, class F>
__device__ __forceinline__ void pieces(const Elem<T>* p, int n, F f) {
  constexpr int V = 16 / sizeof(Elem<T>), S = kChunkElems / (V * kThreads);
  v4i x[S];
  const auto load = [&](int at) {
    const v4i_any* q = reinterpret_cast<const v4i_any*>(p + at);
    if constexpr (LAST) return __builtin_nontemporal_load(q);
    else return (v4i)*q;
  };
  const auto use = [&](int s, int at) {
    Elem<T> v[V];
    __builtin_memcpy(v, &x[s], 16);
    f(v, V, at);
  };
  if (n == kChunkElems) {
#pragma unroll
    for (int s = 0; s < S; ++s) x[s] = load((s * kThreads + threadIdx.x) * V);
#pragma unroll
    for (int s = 0; s < S; ++s) use(s, (s * kThreads + (int)threadIdx.x) * V);
    return;
  }
  // whole pieces, all of them in flight together; then the values past the last
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int at = (s * kThreads + (int)threadIdx.x) * V;
    if (at + V <= n) x[s] = load(at);
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int at = (s * kThreads + (int)threadIdx.x) * V;
    if (at + V <= n) use(s, at);
  }
  if (n % V && (int)threadIdx.x == n / V % kThreads) {
    Elem<T> v[V];
    const int at = n / V * V;
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = at + e < n ? p[at + e] : (Elem<T>)0.0f;
    f(v, n - at, at);
  }
}

// f on the tensor's type
template <class F>
__device__ __forceinline__ void with_type(int type, F f) {
  if (type == kBF16) f(std::integral_constant<int, kBF16>{});
  else if (type == kF16) f(std::integral_constant<int, kF16>{});
  else f(std::integral_constant<int, kF32>{});
}

// The sum of every thread's value, in every thread.
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double red[kThreads / 64];
#pragma unroll
  for (int d = 32; d; d /= 2) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x / 64] = s;
  __syncthreads();
  s = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) s += red[w];
  return s;
}

__global__ void __launch_bounds__(kThreads) k_grad_squares(Table t, double* part) {
  double s = 0.0;
  chunks(t, Run(t, false), false, [&](int i, int64_t e0, int n, int type) {
    with_type(type, [&](auto tc) {
      constexpr int T = decltype(tc)::value;
      pieces<T, false>(static_cast<const Elem<T>*>(t.in[i]) + e0, n, [&](const auto& v, int, int) {
#pragma unroll
        for (int e = 0; e < (int)(16 / sizeof(v[0])); ++e) {  // past a tensor's end: zeros
          const double x = (double)(float)v[e];
          s = fma(x, x, s);
        }
      });
    });
  });
  s = block_sum(s);
  if (threadIdx.x == 0) part[t.part0 + blockIdx.x] = s;
}

__device__ __forceinline__ double norm_of(const double* part, int parts) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  return sqrt(block_sum(s));
}

__global__ void __launch_bounds__(kThreads) k_grad_norm(const double* part, int parts, float* norm) {
  const double v = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = (float)v;
}

__global__ void __launch_bounds__(kThreads) k_grad_scale(Table t, const double* part, int parts, float max_norm,
                                                         float* norm) {
  const Run run(t, true);  // on its way while the norm is added up
  const double v = norm_of(part, parts);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  // (a NaN norm gives NaN, an infinite one 0)  The factor and its products are f64, which
  // has the range for any of them: rounded to f32 first, the factor would bring as much
  // error as the product's own rounding, and more below f32's normal range.
  const double q = max_norm / (v + 1e-6), c = q > 1.0 ? 1.0 : q;
  chunks(t, run, true, [&](int i, int64_t e0, int n, int type) {
    if (c == 1.0 && t.in[i] == t.out[i]) return;  // nothing to change
    with_type(type, [&](auto tc) {
      constexpr int T = decltype(tc)::value;
      using E = Elem<T>;
      E* out = static_cast<E*>(t.out[i]) + e0;
      pieces<T, true>(static_cast<const E*>(t.in[i]) + e0, n, [&](const auto& v, int m, int at) {
        constexpr int V = 16 / sizeof(E);
        E x[V];
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = (E)(float)((double)(float)v[e] * c);
        if (m == V) {
          v4i w;
          __builtin_memcpy(&w, x, 16);
          __builtin_nontemporal_store(w, reinterpret_cast<v4i_any*>(out + at));
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (e < m) out[at + e] = x[e];
        }
      });
    });
  });
}

int launches(int count) { return (count + kTable - 1) / kTable; }

// The chunks of a tensor.
uint64_t chunks_of(const GradTensor& g) { return ((uint64_t)g.n + kChunkElems - 1) / kChunkElems; }

// Calls f(table, blocks) for each launch; returns the number of partial sums.
template <class F>
int each_table(const GradTensor* g, int count, F f) {
  uint64_t all = 0;
  for (int i = 0; i < count; ++i) all += chunks_of(g[i]);
  int part = 0;
  Table t;
  for (int i = 0; i < count;) {
    uint32_t total = 0;
    t.count = 0;
    for (; i < count && t.count < kTable; ++i) {
      if (!g[i].n) continue;
      const int k = t.count++;
      total += (uint32_t)chunks_of(g[i]);
      t.in[k] = g[i].in;
      t.out[k] = g[i].out;
      t.end[k] = total;
      t.last[k] = (uint32_t)((g[i].n - 1) % kChunkElems + 1) | (uint32_t)g[i].type << 16;
    }
    if (!t.count) break;
    // the launch's share of kBlocks blocks, at least one
    const uint64_t share = all <= kBlocks ? total : (uint64_t)total * kBlocks / all;
    const unsigned blocks = (unsigned)(share ? share : 1);
    t.part0 = part;
    t.each = total / blocks;
    t.more = total % blocks;
    part += (int)blocks;
    f(t, blocks);
  }
  return part;
}

}  // namespace

size_t grad_workspace(int count) { return (size_t)(kBlocks + launches(count)) * sizeof(double); }

hipError_t launch_grad_norm(const GradTensor* g, int count, float* norm, void* ws, hipStream_t st) {
  double* part = static_cast<double*>(ws);
  const int parts = each_table(g, count, [&](const Table& t, unsigned blocks) {
    k_grad_squares<<<blocks, kThreads, 0, st>>>(t, part);
  });
  k_grad_norm<<<1, kThreads, 0, st>>>(part, parts, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradTensor* g, int count, float max_norm, float* norm, void* ws, hipStream_t st) {
  double* part = static_cast<double*>(ws);
  const int parts = each_table(g, count, [&](const Table& t, unsigned blocks) {
    k_grad_squares<<<blocks, kThreads, 0, st>>>(t, part);
  });
  if (!parts) {  // no values: norm 0
    if (norm) k_grad_norm<<<1, kThreads, 0, st>>>(part, 0, norm);
    return hipGetLastError();
  }
  bool first = true;
  each_table(g, count, [&](const Table& t, unsigned blocks) {
    k_grad_scale<<<blocks, kThreads, 0, st>>>(t, part, parts, max_norm, first ? norm : nullptr);
    first = false;
  });
  return hipGetLastError();
}

}  // namespace moe
