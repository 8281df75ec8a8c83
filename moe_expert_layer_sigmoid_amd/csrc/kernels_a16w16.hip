// The whole expert layer for a few tokens on 16-bit experts, in two launches:
//   k_few_up    routing and remap of every token in every block (a token's logits
//               are 1.5 KB in L2, a launch more costs longer); then, for 16
//               columns of F of a touched slot, h = W1 x and
//               act = w_tj silu(gate) up, the token's routing weight folded in, so
//               that the sum over a token's experts needs no second pass;
//   k_few_down  out[t] = sum over the touched slots of W2 act: a block owns a few
//               rows of H for all tokens and all slots, so that sums stay in
//               f32 accumulators from the first slot to the last and nothing is
//               joined in memory.
// act goes from one to the other in f32, and the second product takes it in three
// parts of the operands' type that add up to it, so that no bit and no range of it
// is lost (rounded once to 16 bits, it would bring as much error as the output's own
// rounding: normwise 0.0024 for 0.0017 in bf16; in two 16-bit parts, f16's range ended
// at 65504.  Parted in each block as it is used: both launches for 32 tokens on 48 of
// 384 experts 305 us, f16 307, for 303 with two parts stored).
// MFMA columns are tokens (16 a tile), rows are weight rows.  Bound by the touched
// experts' weights, streamed as ring.hpp says: H 7168, F 2048, bf16, one token on 6
// experts 57 + 32 us (6.2 and 5.4 TB/s), 16 tokens on 43 371 + 190 (6.8 and 6.7).

#include <hip/hip_runtime.h>

#include <math.h>

#include <type_traits>

#include "act_device.hpp"
#include "moe_internal.hpp"
#include "ring.hpp"
#include "route_device.hpp"

namespace moe {

constexpr int kPairs = kFewMaxT * 16;  // T k at most

// The touched slots, ascending; the pairs of an entry are act rows [start, start +
// popc(mask)), one per bit (token) of mask, ascending.  A slot with more than 16 tokens
// is two entries, and its weights are then read twice (H 7168, F 2048, all tokens on
// 8 experts: 16 tokens 131 us, 32 241).
struct FewTable {
  int n;
  int pad[3];
  uint32_t mask[kPairs];
  uint16_t slot[kPairs], start[kPairs];
};

namespace {

// ---- routing: the block's view of all tokens -------------------------------
struct Routed {
  FewTable tab;
  uint8_t tok[kPairs];  // of a row: its token
  float w[kPairs];      // ... and its routing weight
};
struct RouteScratch {
  int phys[kPairs];
  float w[kPairs];
  uint32_t mask[1024];  // of a local slot: its tokens
  int before[1024];     // ... and its index among the touched ones
  int rep_slots[1024];
};

template <int EPL, int W>
__device__ __forceinline__ void route_all(const FewArgs& p, Routed& r, RouteScratch& s) {
  constexpr int kThreads = W * 64, kWaves = W;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.t_dev ? min(max(*p.t_dev, 0), p.T) : p.T;
  const bool flat = p.R_max == 1;  // one replica each: the slots are read beside the logits
  for (int i = tid; i < p.P_local; i += kThreads) s.mask[i] = 0;
  if (flat)
    for (int i = tid; i < p.E; i += kThreads) s.rep_slots[i] = p.rep_slots[i];
  __syncthreads();
  const bool first = blockIdx.x == 0;
  auto keep = [&](int t, int j, int e, float w) {
    int ph;
    e = min(e, p.E - 1);  // (NaN logits, against the contract, may choose past E)
    if (flat) ph = s.rep_slots[e];
    else ph = p.rep_slots[(size_t)e * p.R_max + replica(fmix32(p.base + (uint32_t)t), p.rep_count[e], p.R_max)];
    s.phys[t * p.k + j] = ph;
    s.w[t * p.k + j] = w;
    const int q = ph - p.p0;
    if (q >= 0 && q < p.P_local) atomicOr(&s.mask[q], 1u << t);
    if (first) {
      if (p.ids) p.ids[t * p.k + j] = e;
      if (p.wts) p.wts[t * p.k + j] = w;
      if (p.phys) p.phys[t * p.k + j] = ph;
      if (p.load_hist && ph >= 0 && ph < p.P_total) atomicAdd(&p.load_hist[ph], 1);  // whole numbers: any order
    }
  };
  if (n <= kWaves) {
    if (wave < n) {
      int e;
      float w;
      route64<EPL>(p.logits + (size_t)wave * p.E, p.E, p.k, lane, e, w);
      if (lane < p.k) keep(wave, lane, e, w);
    }
  } else {
    for (int t0 = 0; t0 < n; t0 += kThreads / 16) {
      const int t = t0 + tid / 16;
      int e;
      float w;
      route16<4 * EPL>(p.logits + (size_t)min(t, n - 1) * p.E, p.E, p.k, tid & 15, e, w);
      if (t < n && (tid & 15) < p.k) keep(t, tid & 15, e, w);
    }
  }
  if (first && p.phys)
    for (int i = n * p.k + tid; i < p.T * p.k; i += kThreads) p.phys[i] = -1;
  __syncthreads();
  if (wave == 0) {  // the touched slots and their rows, 64 slots at a time
    int nt = 0, rows = 0;
    for (int c = 0; c < p.P_local; c += 64) {
      const uint32_t m = c + lane < p.P_local ? s.mask[c + lane] : 0;
      const int np = __popc(m);
      int pre = np | (np > 16 ? 2 : np > 0 ? 1 : 0) << 16;  // pairs, and entries above them
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(pre, d);
        if (lane >= d) pre += up;
      }
      if (m) {
        const int end = nt + (pre >> 16), i = end - (np > 16 ? 2 : 1), r0 = rows + (pre & 0xFFFF) - np;
        uint32_t rest = m;  // without its first 16 tokens
#pragma unroll 1
        for (int k = 0; k < 16; ++k) rest &= rest - 1;
        s.before[c + lane] = i;
        r.tab.slot[i] = (uint16_t)(c + lane);
        r.tab.start[i] = (uint16_t)r0;
        r.tab.mask[i] = m ^ rest;
        if (rest) {
          r.tab.slot[i + 1] = (uint16_t)(c + lane);
          r.tab.start[i + 1] = (uint16_t)(r0 + 16);
          r.tab.mask[i + 1] = rest;
        }
      }
      const int all = __builtin_amdgcn_readlane(pre, 63);
      nt += all >> 16;
      rows += all & 0xFFFF;
    }
    if (lane == 0) r.tab.n = nt;
  }
  __syncthreads();
  // a row's token and weight (the sum, should two of a token's experts share a slot)
  for (int i = tid; i < n * p.k; i += kThreads) {
    const int t = i / p.k, q = s.phys[i] - p.p0;
    if (q < 0 || q >= p.P_local) continue;
    const int b = s.before[q], row = r.tab.start[b] + __popc(s.mask[q] & ((1u << t) - 1));
    float w = 0.0f;
    for (int j = 0; j < p.k; ++j)
      if (s.phys[t * p.k + j] == s.phys[i]) w += s.w[t * p.k + j];
    r.tok[row] = (uint8_t)t;
    r.w[row] = w;
  }
  __syncthreads();
}

template <int TY, int EPL, int W>
__global__ void __launch_bounds__(W * 64, 2) k_few_up(FewArgs p, int ncnt) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kThreads = W * 64, kWaves = W;
  using R = Ring<TY, 2, 1>;
  __shared__ __align__(1024) uint8_t ring[kWaves * kRingBytes];
  __shared__ __align__(16) float red[kWaves][2][256];
  __shared__ Routed r;
  static_assert(sizeof(RouteScratch) <= sizeof(ring), "scratch in the ring");
  route_all<EPL, W>(p, r, *reinterpret_cast<RouteScratch*>(ring));
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, q = lane >> 4;
  if (blockIdx.x == 0) {
    const int m = r.tab.n;
    for (int i = tid; i < ncnt; i += kThreads) p.cnt[i] = 0;
    if (tid == 0) p.tab->n = m;
    for (int i = tid; i < m; i += kThreads) {
      p.tab->slot[i] = r.tab.slot[i];
      p.tab->start[i] = r.tab.start[i];
      p.tab->mask[i] = r.tab.mask[i];
    }
  }
  // Items: 16 columns of an entry, dealt to the blocks in turn.  (Equal shares to the
  // column, the last part of a block's narrower, were slower: 388 us for 371 at
  // 43 slots, 60 for 57 at 6.  A narrow part has as many stages, of fewer bytes in flight.)
  const int H = p.H, F = p.F, nct = F / 16;
  const int items = __builtin_amdgcn_readfirstlane(r.tab.n) * nct;
  if ((int)blockIdx.x >= items) return;  // fewer slots touched than pairs: the same in the whole block
  const int kst = H / kStageK;
  const int rounds = (kst + kWaves * R::NS - 1) / (kWaves * R::NS);
  const uint32_t rowb = 2u * (uint32_t)H;
  const uint32_t avo = (uint32_t)(lane >> 3) * rowb + dma_piece(lane);
  const rsrc_t xr = make_rsrc(p.x, (uint32_t)p.T * rowb), none = make_rsrc(p.x, 0);

  // where the next loads come from
  int item = blockIdx.x, round = 0;
  rsrc_t wr = none;
  uint32_t wso = 0, xvo = kOob;
  auto seek = [&]() {
    const bool live = item < items;
    const int i = live ? item / nct : 0, ct = live ? item - i * nct : 0;
    const int slot = __builtin_amdgcn_readfirstlane((int)r.tab.slot[i]);
    const int start = r.tab.start[i], n = live ? __popc(r.tab.mask[i]) : 0;
    wr = make_rsrc(static_cast<const uint8_t*>(p.w1) + (size_t)slot * 2 * F * rowb, live ? 2u * (uint32_t)F * rowb : 0u);
    wso = (uint32_t)ct * 16u * rowb;
    xvo = l16 < n ? (uint32_t)r.tok[start + l16] * rowb + 16u * q : kOob;
  };
  R g;
  auto issue = [&](lds_u8* to, int u) __attribute__((always_inline)) {
    const int st = wave + kWaves * (R::NS * round + u);
    const bool live = st < kst;
    const uint32_t so = (uint32_t)st * 128u;
    const rsrc_t a = live ? wr : none, x = live ? xr : none;
#pragma unroll
    for (int m = 0; m < 4; ++m)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(a, (lds_void)(to + u * R::kSlot + m * 1024), 16, avo,
                                               so + wso + ((m & 1) * 8u + (m >> 1) * (uint32_t)F) * rowb, 0, 2);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) g.b[u][0][kk] = buf_load16(x, xvo, so + 64u * kk);
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
          item += gridDim.x;
          seek();
        }
      }
      issue(to, (u + R::PRE) % R::NS);
      consume(from + u * R::kSlot, g, u);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  lds_u8* const mine = (lds_u8*)ring + wave * kRingBytes;
  const auto clear = [&]() { g.acc[0][0] = g.acc[1][0] = v4f{0.f, 0.f, 0.f, 0.f}; };
  const auto finish = [&](int it) {
    const int i = it / nct, ct = it - i * nct;
    const int start = r.tab.start[i], np = __popc(r.tab.mask[i]);
    const v4f v[2] = {g.acc[0][0], g.acc[1][0]};
    float s[2];
    reduce<2, W>(red, v, s);
    const int j = tid / 16;  // (np <= 16: the first four waves)
    if (j < np) {
      const float gate[1] = {s[0]}, up[1] = {s[1]};
      float y[1];
      act_row<kActSilu>(gate, up, y);
      p.act[(size_t)(start + j) * F + ct * 16 + tid % 16] = y[0] * r.w[start + j];
    }
  };
  if (const int per = (kst + kWaves - 1) / kWaves; per <= R::PRE) {  // short: one burst an item
    for (; item < items; item += gridDim.x) {
      clear();
      seek();
      burst<R>(mine, per, issue, [&](const lds_u8* from, int u) { consume(from, g, u); });
      finish(item);
    }
    return;
  }
  seek();
  int it = blockIdx.x;  // the item being added up
  for (int n = -1;; ++n) {
    if (n <= 0) clear();
    stages(mine, mine, n < 0);
    if (n + 1 < rounds) continue;
    finish(it);
    it += gridDim.x;
    if (it >= items) break;
    n = -1;  // the next item's first stages are on their way
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the block
#endif
}

// ---- f32 operands of 16-bit matrix instructions -----------------------------
// The largest of a value over the four lanes l16 + 16 q, in each of them.
__device__ __forceinline__ float max_of_quads(float m) {
  const uint32_t a = __float_as_uint(m);
  const auto x = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  const uint32_t b = __float_as_uint(fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])));
  const auto y = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
}

// Eight finite values (or NaN) as parts[0] + parts[1] + parts[2], each truncated to
// its bits: 24 bits are 8 + 8 + 8 of bf16, 11 + 11 + 2 of f16.  Parts of f16 end at 2^-24.
template <int TY>
__device__ __forceinline__ void split(const float (&v)[8], v4i (&parts)[3]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    float a = v[e], b = v[e + 1];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if constexpr (TY == kBF16) {
        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
        parts[k][e / 2] = (int)__builtin_amdgcn_perm(ub, ua, 0x07060302u);
        if (k < 2) {
          a -= __uint_as_float(ua & 0xFFFF0000u);
          b -= __uint_as_float(ub & 0xFFFF0000u);
        }
      } else {
        const auto h = __builtin_amdgcn_cvt_pkrtz(a, b);
        parts[k][e / 2] = __builtin_bit_cast(int, h);
        if (k < 2) {
          a -= (float)h[0];
          b -= (float)h[1];
        }
      }
    }
  }
}

// hr <= 16 NA: rows of H a block.  Few rows of H leave compute units idle: zs blocks
// then share a block's entries, as far as every wave gets kLeast stages (17 tokens, H 640,
// F 1024, 9 of 15 experts: 9.6 us with 2 or 3, 12.6 with 4, past one burst); each stores its
// f32 sums, and the last of them to finish (a counter, zeroed by k_few_up) adds
// them in order.  The sums are stored and loaded device-coherent, past the
// dies' own L2s, so that completion is all that has to be waited for.
constexpr int kDownWaves = 8;
constexpr int kLeast = 2;
template <int TY, int NA, int NT>
__global__ void __launch_bounds__(kDownWaves * 64, 2) k_few_down(FewArgs p, int hr, int zs) {
#ifdef __HIP_DEVICE_COMPILE__
  using R = Ring<TY, NA, NT, 2>;
  constexpr int W = kDownWaves;
  __shared__ __align__(1024) uint8_t ring[W * kRingBytes];
  __shared__ __align__(16) float red[W][NA][256];
  __shared__ FewTable tab;
  __shared__ bool s_last;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, q = lane >> 4;
  const int nt = p.tab->n;
  const int H = p.H, F = p.F, kst = F / kStageK;
  const int total = nt * kst;  // stages of all entries in a row
  const int parts = max(1, min(zs, (total + kLeast * W - 1) / (kLeast * W)));
  const int tile = blockIdx.x / zs, z = blockIdx.x % zs;
  if (z >= parts) return;
  for (int i = tid; i < nt; i += W * 64) {
    tab.slot[i] = p.tab->slot[i];
    tab.start[i] = p.tab->start[i];
    tab.mask[i] = p.tab->mask[i];
  }
  __syncthreads();
  const int h0 = tile * hr, nh = min(hr, H - h0);
  const int each = (total + parts - 1) / parts, first = z * each, end = min(total, first + each);
  const int rounds = (each + W * R::NS - 1) / (W * R::NS);
  const uint32_t rowb = 2u * (uint32_t)F, actb = 4u * (uint32_t)F;
  uint32_t avo[2 * NA];
#pragma unroll
  for (int m = 0; m < 2 * NA; ++m)
    avo[m] = (lane >> 3) + 8 * m < nh ? (uint32_t)((lane >> 3) + 8 * m) * rowb + dma_piece(lane) : kOob;
  const rsrc_t ar = make_rsrc(p.act, (uint32_t)(p.T * p.k) * actb), none = make_rsrc(p.act, 0);

  int at = first + wave;          // the next loads: stage of all,
  int i = at / kst, s = at % kst;  // entry, stage of it
  rsrc_t wr = none;
  uint32_t bvo[NT], on = 0, held = 0;  // on: bit c: entry i has the lane's token of tile c; held: of each stage in the ring
  auto seek = [&]() {  // of entry i
    const bool live = i < nt;
    const int ii = live ? i : 0;
    const int slot = __builtin_amdgcn_readfirstlane(live ? (int)tab.slot[ii] : 0);
    const uint32_t mask = live ? tab.mask[ii] : 0;
    const int start = live ? tab.start[ii] : 0;
    wr = make_rsrc(static_cast<const uint8_t*>(p.w2) + ((size_t)slot * H + h0) * rowb, live ? (uint32_t)nh * rowb : 0u);
    on = 0;
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      const int t = 16 * c + l16;
      on |= (mask >> t & 1) << c;
      bvo[c] = mask >> t & 1 ? (uint32_t)(start + __popc(mask & ((1u << t) - 1))) * actb + 32u * q : kOob;
    }
  };
  R g;
#pragma unroll
  for (int a = 0; a < NA; ++a)
#pragma unroll
    for (int c = 0; c < NT; ++c) g.acc[a][c] = v4f{0.f, 0.f, 0.f, 0.f};
  if (first < end) {
    seek();
    auto issue = [&](lds_u8* to, int u) __attribute__((always_inline)) {
      const uint32_t so = (uint32_t)s * 128u;
      const bool live = at < end;
      const rsrc_t w = live ? wr : none, b = live ? ar : none;
#pragma unroll
      for (int m = 0; m < 2 * NA; ++m)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(w, (lds_void)(to + u * R::kSlot + m * 1024), 16, avo[m], so, 0, 2);
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          g.b[u][2 * c][kk] = buf_load16(b, bvo[c], 2 * so + 128u * kk);
          g.b[u][2 * c + 1][kk] = buf_load16(b, bvo[c] + 16u, 2 * so + 128u * kk);  // (kOob + 16: still past every buffer)
        }
      held = (held & ~(((1u << NT) - 1) << (u * NT))) | on << (u * NT);
      at += W;
      if ((s += W) >= kst) {
        i += s / kst;
        s %= kst;
        seek();
      }
    };
    // A stage's products, in sums of their own, which the tokens that its expert does not
    // see leave out (zeros times a weight that is not finite would be NaN).  f16: a
    // token's 64 values are scaled by the power of two that brings the largest
    // to [2^14, 2^15), so that its range holds them; what its parts cannot hold is below
    // 2^-38 of that one.
    auto eat = [&](const lds_u8* from, int u) __attribute__((always_inline)) {
      const auto weights = [&](int a, int kk) {
        return *reinterpret_cast<const lds_v4i*>(from + a * 2048 + l16 * 128 + (((4 * kk + q) ^ (l16 & 7)) * 16));
      };
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        const bool see = held >> (u * NT + c) & 1;
        if (NT > 1 && !__ballot(see)) continue;  // none of the tile's tokens (the 305 us above were 312)
        const auto largest = [&]() {
          float m = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(__int_as_float(g.b[u][2 * c + i / 4 % 2][i / 8][i % 4])));
          return m;
        };
        v4f sum[NA];
#pragma unroll
        for (int a = 0; a < NA; ++a) sum[a] = v4f{0.f, 0.f, 0.f, 0.f};
        float m = largest();
        if (__ballot(m == INFINITY)) {  // infinities have no second part: their products apart
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            v4i inf = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int v = g.b[u][2 * c + e / 4][kk][e % 4];
              const bool is = (v & 0x7FFFFFFF) == 0x7F800000;
              const uint32_t h = (uint32_t)v >> 31 << 15 | (TY == kBF16 ? 0x7F80u : 0x7C00u);
              inf[e / 2] |= is ? (int)(h << (e % 2 * 16)) : 0;
              g.b[u][2 * c + e / 4][kk][e % 4] = is ? 0 : v;
            }
#pragma unroll
            for (int a = 0; a < NA; ++a) sum[a] = mfma16<TY>(weights(a, kk), inf, sum[a]);
          }
          m = largest();
        }
        float scale = 1.0f, back = 1.0f;
        if (TY == kF16) {
          const uint32_t e = max(__float_as_uint(max_of_quads(m)) >> 23, 15u);  // m = 2^(e - 127) to twice that
          scale = __uint_as_float((268u - e) << 23);
          back = __uint_as_float((e - 14u) << 23);
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          float v[8];
          v4i part[3];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __int_as_float(g.b[u][2 * c + e / 4][kk][e % 4]) * scale;
          split<TY>(v, part);
#pragma unroll
          for (int a = 0; a < NA; ++a) {
            const v4i w = weights(a, kk);
#pragma unroll
            for (int k = 2; k >= 0; --k) sum[a] = mfma16<TY>(w, part[k], sum[a]);
          }
        }
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float old = g.acc[a][c][e];
            g.acc[a][c][e] = see ? fmaf(sum[a][e], back, old) : old;
          }
      }
    };
    auto stages = [&](lds_u8* __restrict__ to, const lds_u8* __restrict__ from, bool first) __attribute__((always_inline)) {
      if (first) {
#pragma unroll
        for (int u = 0; u < R::PRE; ++u) issue(to, u);
        return;
      }
#pragma unroll
      for (int u = 0; u < R::NS; ++u) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"((R::PRE - 1) * R::I) : "memory");
        __builtin_amdgcn_sched_barrier(0);
        issue(to, (u + R::PRE) % R::NS);
        eat(from + u * R::kSlot, u);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    lds_u8* const mine = (lds_u8*)ring + wave * kRingBytes;
    if (const int per = (each + W - 1) / W; per <= R::PRE) {
      burst<R>(mine, per, issue, eat);
    } else {
      for (int n = -1; n < rounds; ++n) stages(mine, mine, n < 0);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the block
    }
  }
  const auto put = [&](int t, int h, float v) { static_cast<Half<TY>*>(p.out)[(size_t)t * H + h0 + h] = (Half<TY>)v; };
  float* const part = p.part + (size_t)h0 + (size_t)z * p.T * H;
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    v4f v[NA];
    float o[NA];
#pragma unroll
    for (int a = 0; a < NA; ++a) v[a] = g.acc[a][c];
    reduce<NA, W>(red, v, o);
    const int t = 16 * c + tid / 16;
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int h = 16 * a + tid % 16;
      if (tid < 256 && t < p.T && h < nh) {
        if (parts == 1) put(t, h, o[a]);
        else __hip_atomic_store(part + (size_t)t * H + h, o[a], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }
  if (parts == 1) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0)
    s_last = __hip_atomic_fetch_add(p.cnt + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
  __syncthreads();
  if (!s_last) return;
  for (int e = tid; e < p.T * nh; e += W * 64) {
    const int t = e / nh, h = e % nh;
    const float* const o = p.part + (size_t)t * H + h0 + h;
    float v = 0.0f;
    for (int k = 0; k < parts; k += 8) {
      float x[8];
#pragma unroll
      for (int m = 0; m < 8; ++m)
        x[m] = __hip_atomic_load(o + (size_t)min(k + m, parts - 1) * p.T * H, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int m = 0; m < 8; ++m)
        if (k + m < parts) v += x[m];
    }
    put(t, h, v);
  }
#endif
}

// How k_few_down is divided: rows of H a block, blocks that share an entry's
// reduction.  From 2048 rows on, what gives every compute unit one block; below,
// tiles of 16 rows (32 for two tiles of tokens) and as many blocks a tile as fill the card.
struct DownPlan {
  int hr, tiles, zs;
};
DownPlan down_plan(int T, int H) {
  const int whole = T > 16 ? 32 : 16, fit = (H + kCus - 1) / kCus;
  DownPlan d;
  d.zs = kCus / ((H + whole - 1) / whole);
  if (d.zs < 2) d.zs = 1;
  d.hr = d.zs > 1 ? whole : fit < 32 ? fit : 32;
  d.tiles = (H + d.hr - 1) / d.hr;
  return d;
}

template <int TY>
hipError_t run(const FewArgs& p, hipStream_t st) {
  const long slots = (long)p.P_local * (p.T > 16 ? 2 : 1), pairs = (long)p.T * p.k;
  const long most = (slots < pairs ? slots : pairs) * (p.F / 16);
  const DownPlan d = down_plan(p.T, p.H);
  const auto up = [&](auto epl, auto w) {
    constexpr int EPL = decltype(epl)::value, W = decltype(w)::value, kMost = 2 * kCus * kRingWaves / W;
    k_few_up<TY, EPL, W><<<(unsigned)(most < kMost ? most : kMost), W * 64, 0, st>>>(p, d.tiles);
  };
  const auto up_w = [&](auto w) {
    if (p.E <= 128) up(std::integral_constant<int, 2>{}, w);
    else if (p.E <= 384) up(std::integral_constant<int, 6>{}, w);
    else up(std::integral_constant<int, 16>{}, w);
  };
  // Eight waves a block and one block a compute unit where the items expected (of
  // slots that uniform routing touches) are no more than the units, else four and two.
  const double miss = pow(1.0 - (double)p.k / p.E, p.T);
  if (p.P_local * (1.0 - miss) * (p.F / 16) <= kCus) up_w(std::integral_constant<int, 8>{});
  else up_w(std::integral_constant<int, 4>{});
  const unsigned down = (unsigned)(d.tiles * d.zs);
  if (p.T > 16) k_few_down<TY, 2, 2><<<down, kDownWaves * 64, 0, st>>>(p, d.hr, d.zs);
  else if (d.hr > 16) k_few_down<TY, 2, 1><<<down, kDownWaves * 64, 0, st>>>(p, d.hr, d.zs);
  else k_few_down<TY, 1, 1><<<down, kDownWaves * 64, 0, st>>>(p, d.hr, d.zs);
  return hipGetLastError();
}

}  // namespace

size_t few_table_bytes() { return sizeof(FewTable); }

// (for any T up to T_max, which has the most rows but not always the most blocks a tile)
size_t few_sums_bytes(int T_max, int H) {
  size_t n = 0;
  for (int T = 1; T <= T_max && T <= kFewMaxT; ++T) {
    const DownPlan d = down_plan(T, H);
    const size_t m = d.zs > 1 ? (size_t)d.zs * T * H * sizeof(float) : 0;
    n = m > n ? m : n;
  }
  return n;
}

hipError_t launch_few(int type, const FewArgs& p, hipStream_t st) {
  return type == kBF16 ? run<kBF16>(p, st) : run<kF16>(p, st);
}

}  // namespace moe
