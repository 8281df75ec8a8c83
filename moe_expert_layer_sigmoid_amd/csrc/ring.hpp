// The weight stream of the kernels for few token rows: a block of four or eight waves
// takes 16 weight rows (or twice that), each wave every fourth or eighth 128-byte piece of
// the reduction.  The weights come by DMA, in whole lines, into an LDS ring that
// belongs to one wave alone: no wave waits for another but at the end of a
// block's rows, and the next rows' weights are then already on their way.  The token
// operand (a few KB, from L2) is loaded straight into registers as far ahead.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_kernel.hpp"

namespace moe {
namespace {

constexpr int kRingWaves = 4;      // of a block, two blocks a compute unit; or eight, one block
constexpr int kRingBytes = 16384;  // of a wave
constexpr int kStageK = 64;        // reduction elements of a stage: 128 bytes of a row

template <int TY>
using Half = std::conditional_t<TY == kBF16, __bf16, _Float16>;

// A wave's ring: NA tiles of 16 weight rows a stage, NS stages, and the token
// operands of those stages in registers: NT tiles of 16 tokens, a lane's eight values
// of an MFMA in P words of 16 bytes.
template <int TY, int NA, int NT, int P = 1>
struct Ring {
  static constexpr int kSlot = NA * 2048;
  static constexpr int NS = kRingBytes / kSlot, PRE = NS - 1;
  static constexpr int I = 2 * NA + 2 * NT * P;  // loads of a stage
  static_assert((PRE - 1) * I < 63, "vmcnt range");
  v4i b[NS][NT * P][2];
  v4f acc[NA][NT];
};

// ---- one stage --------------------------------------------------------------
// Lane offsets of the DMA: 8 rows of 128 bytes an instruction, the 16-byte pieces
// of a row permuted so that the reads spread over the LDS banks.
__device__ __forceinline__ uint32_t dma_piece(int lane) { return 16u * (uint32_t)((lane & 7) ^ (lane >> 3)); }

template <int TY, int NA, int NT>
__device__ __forceinline__ void consume(const lds_u8* rd, Ring<TY, NA, NT>& g, int u) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const v4i w = *reinterpret_cast<const lds_v4i*>(rd + a * 2048 + l16 * 128 + (((4 * kk + q) ^ (l16 & 7)) * 16));
#pragma unroll
      for (int c = 0; c < NT; ++c) g.acc[a][c] = mfma16<TY>(w, g.b[u][c][kk], g.acc[a][c]);
    }
}

// All of a wave's `per` <= PRE stages in one burst: short reductions, where a full
// ring would wait for stages that are not there (two tokens, H 128, F 32, 8 experts:
// 5.5 + 3.4 us in one burst, 6.4 + 8.3 through the ring).
template <class R, class Issue, class Eat>
__device__ __forceinline__ void burst(lds_u8* mine, int per, Issue issue, Eat eat) {
#pragma unroll
  for (int u = 0; u < R::PRE; ++u)
    if (u < per) issue(mine, u);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 0; u < R::PRE; ++u)
    if (u < per) eat(mine + u * R::kSlot, u);
}

// The W waves' sums of acc[a][c], by thread of the first four waves (token column
// tid / 16, weight row tid % 16).
template <int NA, int W>
__device__ __forceinline__ void reduce(float (*red)[NA][256], const v4f (&v)[NA], float (&s)[NA]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int a = 0; a < NA; ++a) *reinterpret_cast<v4f*>(&red[wave][a][(lane & 15) * 16 + 4 * (lane >> 4)]) = v[a];
  // (LDS alone is waited for: the loads of the next stages stay in flight)
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    s[a] = red[0][a][tid % 256];
#pragma unroll
    for (int w = 1; w < W; ++w) s[a] += red[w][a][tid % 256];
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace
}  // namespace moe
