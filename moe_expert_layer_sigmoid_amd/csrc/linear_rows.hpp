// The product with its epilogue for at most 16 rows in all: the weights of the
// groups with rows are streamed once, every sum is finished in its block, nothing
// is joined in memory.  A block takes an equal share of the groups' output columns, 16
// at a time (gated: 16 gate and 16 up columns); W waves a block: eight, one block a
// compute unit, where that gives a unit 16 columns at most, else four and two.  Bound by the weights and by
// the latency of one burst.  (One row, 4096 x 7168, gated: 13.1 us, 18.0 by a block's
// eight waves loading weights into registers; 512 x 7168 plain 8.5 and 11.0; 1024 x
// 1024 gated 4.2, by tiles 7.6.  More rows a group read x too often for that: 48 rows,
// 4096 x 7168 gated, took 25.6 against 17.8 by tiles.)
#pragma once

#include "ring.hpp"

namespace moe {
namespace {

constexpr int kRowsMax = 16;
constexpr int kRowsLeastCols = 4;  // of a block

// BIG: the weights pass the caches (the streaming policy, as in k_linear)
template <int IN, int EP, bool BIG, int W>
__global__ void __launch_bounds__(W * 64, 2) k_linear_rows(LinearArgs p, int out_type) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int G = EP == kGated ? 2 : 1;
  using R = Ring<IN, G, 1>;
  using B = Half<IN>;
  __shared__ __align__(1024) uint8_t ring[W * kRingBytes];
  __shared__ __align__(16) float red[W][G][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, q = lane >> 4;
  const int n_out = p.N / G;
  const RowTiles<kRowsMax> rt(p.off, p.groups, p.rows);  // a tile is a group with rows
  const int cols = rt.total * n_out;
  const int share = max(kRowsLeastCols, (cols + (int)gridDim.x - 1) / (int)gridDim.x);
  int at = blockIdx.x * share;  // of the columns being added up
  const int end = min(cols, at + share);
  if (at >= end) return;
  const uint32_t rowb = 2u * (uint32_t)p.K;
  const int kst = (int)((rowb + 127) / 128);
  const int rounds = (kst + W * R::NS - 1) / (W * R::NS);

  // Columns [c0, c0 + n) of a group and its rows, from column `col` of the row.
  struct Part {
    int g, c0, n, r0, nr;
  };
  auto part = [&](int col) {
    int g, t, lo, hi;
    rt.find(col / n_out, g, t, lo, hi);
    const int c0 = col % n_out;
    return Part{g, c0, min(16, min(n_out - c0, end - col)), lo, hi - lo};
  };

  const rsrc_t none = make_rsrc(p.a, 0);
  int next = at, round = 0;  // the next loads
  rsrc_t wr = none, xr = none;
  // Row offsets of the DMA instructions: 8 rows each, then the up columns.
  const uint32_t kpc = dma_piece(lane);
  uint32_t avo[2 * G];
  const uint32_t xvo = (uint32_t)l16 * rowb + 16u * q;
  int len = 0;
  auto seek = [&]() {
    const bool live = next < end;
    const Part x = part(live ? next : at);
    len = x.n;
    wr = make_rsrc(static_cast<const uint8_t*>(p.a) + ((size_t)x.g * p.N + x.c0) * rowb, live ? (uint32_t)(p.N - x.c0) * rowb : 0u);
    xr = make_rsrc(static_cast<const uint8_t*>(p.b) + (size_t)x.r0 * rowb, live ? (uint32_t)x.nr * rowb : 0u);
#pragma unroll
    for (int m = 0; m < 2 * G; ++m) {
      const int row = (m & 1) * 8 + (lane >> 3);
      avo[m] = row < x.n ? (uint32_t)(row + (m >> 1) * n_out) * rowb + kpc : kOob;
    }
  };
  R g;
  auto issue = [&](lds_u8* to, int u) __attribute__((always_inline)) {
    const uint32_t so = (uint32_t)(wave + W * (R::NS * round + u)) * 128u;
    const bool in = so + kpc < rowb;  // not so for pieces past the row's end and stages past the last
#pragma unroll
    for (int m = 0; m < 2 * G; ++m)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (lds_void)(to + u * R::kSlot + m * 1024), 16, in && avo[m] != kOob ? avo[m] + so : kOob, 0, 0,
                                               BIG ? 2 : 0);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
      g.b[u][0][kk] = buf_load16(xr, so + 64u * kk + 16u * q < rowb ? xvo + so + 64u * kk : kOob, 0);
  };
  // NS stages; before the first, the loads alone.  to and from are the same ring,
  // as __restrict__: the compiler then places no wait of its own between a DMA in
  // flight and the reads of another stage.
  auto stages = [&](lds_u8* __restrict__ to, const lds_u8* __restrict__ from, bool first) __attribute__((always_inline)) {
    if (first) {
#pragma unroll
      for (int u = 0; u < R::PRE; ++u) issue(to, u);
      return;
    }
#pragma unroll
    for (int u = 0; u < R::NS; ++u) {
      // stage u has landed; the reads of the stage before are done, whose slot is loaded next
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"((R::PRE - 1) * R::I) : "memory");
      __builtin_amdgcn_sched_barrier(0);
      if (u == 1) {  // the loads enter the next round
        if (++round == rounds) {
          round = 0;
          next += len;
          seek();
        }
      }
      issue(to, (u + R::PRE) % R::NS);
      consume(from + u * R::kSlot, g, u);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  lds_u8* const mine = (lds_u8*)ring + wave * kRingBytes;
  const auto clear = [&]() {
#pragma unroll
    for (int a = 0; a < G; ++a) g.acc[a][0] = v4f{0.f, 0.f, 0.f, 0.f};
  };
  // what the epilogue adds, on its way during the product: as it lies in memory, so
  // that nothing waits for it before `finish`
  uint32_t bias[G] = {}, res = 0;
  const auto ahead = [&](const Part& x) {
    const int j = tid / 16, col = x.c0 + tid % 16;
    if (j >= x.nr || tid % 16 >= x.n) return;
    const size_t o = (size_t)(x.r0 + j) * n_out + col;
    if (p.bias) {
#pragma unroll
      for (int h = 0; h < G; ++h) bias[h] = static_cast<const uint16_t*>(p.bias)[(size_t)x.g * p.N + h * n_out + col];
    }
    if (p.res) res = out_type == kF32 ? static_cast<const uint32_t*>(p.res)[o] : static_cast<const uint16_t*>(p.res)[o];
  };
  const auto finish = [&](const Part& x) {
    const int j = tid / 16, col = x.c0 + tid % 16;
    const bool here = j < x.nr && tid % 16 < x.n;  // (nr <= 16: the first four waves)
    const size_t row = (size_t)(x.r0 + j), o = row * n_out + col;
    const auto value = [](uint32_t w) { return (float)__builtin_bit_cast(B, (uint16_t)w); };
    v4f v[G];
    float z[G], y[1];
#pragma unroll
    for (int a = 0; a < G; ++a) v[a] = g.acc[a][0];
    reduce<G, W>(red, v, z);
    auto put = [&](void* out, size_t i, float e) {
      if (out_type == kF32) static_cast<float*>(out)[i] = e;
      else static_cast<B*>(out)[i] = (B)e;
    };
    if (here) {
#pragma unroll
      for (int h = 0; h < G; ++h) {
        z[h] += value(bias[h]);
        if (p.pre) put(p.pre, row * p.N + h * n_out + col, z[h]);
      }
      const float gate[1] = {z[0]}, up[1] = {G == 2 ? z[G - 1] : 1.0f};
      with_act(p.act, [&](auto a) { act_row<decltype(a)::value>(gate, up, y); });
      put(p.out, o, y[0] + (out_type == kF32 ? __uint_as_float(res) : value(res)));
    }
  };
  if (const int per = (kst + W - 1) / W; per <= R::PRE) {  // short: one burst a part
    while (at < end) {
      const Part x = part(at);
      clear();
      next = at;
      seek();
      ahead(x);
      burst<R>(mine, per, issue, [&](const lds_u8* from, int u) { consume(from, g, u); });
      finish(x);
      at += x.n;
    }
    return;
  }
  seek();
  Part x = part(at);
  ahead(x);
  for (int n = -1;; ++n) {
    if (n <= 0) clear();
    stages(mine, mine, n < 0);
    if (n + 1 < rounds) continue;
    finish(x);
    at += x.n;
    if (at >= end) break;
    x = part(at);
    ahead(x);
    n = -1;  // the next columns' first stages are on their way
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the block
#endif
}

}  // namespace
}  // namespace moe
