// Top-k routing of a token by a wavefront or a 16-lane row, shared by the layer's
// front kernels and the few-token layer on 16-bit experts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// ---------------------------------------------------------------------------
// a1 route.  Each of the k rounds takes the argmax of the token's logits
// (largest logit, lower id on ties) and retires the winner's entry (set to
// -inf; inputs are finite).  Weights: sigmoid of the chosen logits over their
// sum, in f32, the sum being a DPP tree over the lanes j < k that hold choice j.
//  - route64, one wavefront per token (the fused small-M front, where the
//    chain's latency counts): lane l holds logits l, l + 64, ...; a round is a
//    scan of the lane's own entries, a DPP reduction inside each 16-lane row
//    and a scalar pick among the four row winners (read with readlane).
//  - route16, one 16-lane row per token, four tokens per wavefront (the
//    standalone routing pass over many tokens, where throughput counts):
//    lane l of the row holds logits l, l + 16, ...; the DPP reduction inside
//    the row leaves the winner in every lane, with no cross-row step.  On the
//    prefill share of 65,536 tokens (384 experts, top-6) it took about 1 %
//    off the forward; in the fused front its longer per-lane scan cost
//    1-2 us at one token.
// Both give the same choices and weights bit for bit (the same comparisons,
// and the weights' sum in the same order, lane 0's tree).
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
  return __int_as_float(dpp<CTRL>(__float_as_int(v)));
}
constexpr int kRor8 = 0x128, kRor4 = 0x124, kQuadSwap2 = 0x4E, kQuadSwap1 = 0xB1;

__device__ __forceinline__ bool better(float av, int ai, float bv, int bi) {
  return av > bv || (av == bv && ai < bi);
}

// (bv, bi) <- the better of itself and its DPP partner's.
template <int CTRL>
__device__ __forceinline__ void take_better(float& bv, int& bi) {
  const float ov = dppf<CTRL>(bv);
  const int oi = dpp<CTRL>(bi);
  const bool take = better(ov, oi, bv, bi);
  bv = take ? ov : bv;
  bi = take ? oi : bi;
}

template <int CTRL>
__device__ __forceinline__ float add_partner(float v) {
  return v + dppf<CTRL>(v);
}

// Route one token per wavefront (`row`: its logits).  Lane j < k returns
// choice j and its weight.
template <int EPL>
__device__ __forceinline__ void route64(const float* __restrict__ row, int E, int k, int lane, int& my_id,
                                        float& my_w) {
  float v[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < E ? row[e] : -INFINITY;
  }
  my_id = 0;
  float my_l = 0.0f;
  for (int j = 0; j < k; ++j) {
    float bv = v[0];
    int bi = lane;
#pragma unroll
    for (int i = 1; i < EPL; ++i) {
      const bool t = v[i] > bv;  // ascending ids: strict > keeps the lower id
      bv = t ? v[i] : bv;
      bi = t ? lane + 64 * i : bi;
    }
    take_better<kRor8>(bv, bi);
    take_better<kRor4>(bv, bi);
    take_better<kQuadSwap2>(bv, bi);
    take_better<kQuadSwap1>(bv, bi);
    float sv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bv), 0));
    int si = __builtin_amdgcn_readlane(bi, 0);
#pragma unroll
    for (int r = 1; r < 4; ++r) {
      const float rv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bv), 16 * r));
      const int ri = __builtin_amdgcn_readlane(bi, 16 * r);
      if (better(rv, ri, sv, si)) {
        sv = rv;
        si = ri;
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = (lane + 64 * i == si) ? -INFINITY : v[i];
    if (lane == j) {
      my_id = si;
      my_l = sv;
    }
  }
  const float s = lane < k ? 1.0f / (1.0f + expf(-my_l)) : 0.0f;
  float sum = add_partner<kRor8>(s);
  sum = add_partner<kRor4>(sum);
  sum = add_partner<kQuadSwap2>(sum);
  sum = add_partner<kQuadSwap1>(sum);
  sum = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sum), 0));
  my_w = s / sum;
}

// Route the token of this lane's 16-lane row (`row`: its logits; EPL logits
// per lane).  Lane l16 < k of the row returns choice l16 and its weight; the
// weights' sum is the row's DPP tree as its lane 0 adds it (the other lanes
// add in other orders), so every choice of the token divides by one value.
template <int EPL>
__device__ __forceinline__ void route16(const float* __restrict__ row, int E, int k, int l16, int& my_id,
                                        float& my_w) {
  float v[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = l16 + 16 * i;
    v[i] = e < E ? row[e] : -INFINITY;
  }
  my_id = 0;
  float my_l = 0.0f;
  for (int j = 0; j < k; ++j) {
    float bv = v[0];
    int bi = l16;
#pragma unroll
    for (int i = 1; i < EPL; ++i) {
      const bool t = v[i] > bv;  // ascending ids: strict > keeps the lower id
      bv = t ? v[i] : bv;
      bi = t ? l16 + 16 * i : bi;
    }
    take_better<kRor8>(bv, bi);
    take_better<kRor4>(bv, bi);
    take_better<kQuadSwap2>(bv, bi);
    take_better<kQuadSwap1>(bv, bi);
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = (l16 + 16 * i == bi) ? -INFINITY : v[i];
    if (l16 == j) {
      my_id = bi;
      my_l = bv;
    }
  }
  const float s = l16 < k ? 1.0f / (1.0f + expf(-my_l)) : 0.0f;
  float sum = add_partner<kRor8>(s);
  sum = add_partner<kRor4>(sum);
  sum = add_partner<kQuadSwap2>(sum);
  sum = add_partner<kQuadSwap1>(sum);
  sum = __shfl(sum, (int)(threadIdx.x & 63) & ~15);
  my_w = s / sum;
}

}  // namespace moe
