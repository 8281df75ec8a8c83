// How a linear product is divided among blocks: block shape, splits of the
// reduction, cache policy and workspace.  Host code alone, without HIP, so that
// the choice for any sizes can be asked for where there is no GPU.
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// moe_type_t of include/moe.h
enum { kBF16 = 0, kF16 = 1, kF32 = 2, kFP8 = 3 };

// What a product computes; "columns" are the output's contiguous dimension.
//  kFwd: y[row, n]  = sum_k x[row, k] w[g, n, k]
//  kDx:  dx[row, k] = sum_n dy[row, n] w[g, n, k]
//  kDw:  dw[g, n, k] = sum over the group's rows of dy[row, n] x[row, k]
enum { kFwd = 0, kDx = 1, kDw = 2 };

struct Plan {
  int nca;       // column tiles
  int nrb;       // row tiles: kDw: of N; else an upper bound over all groups
  int splits;    // ranges of the reduction, each by its own block into its own partial sums
  int sps;       // stages per split (kFwd, kDx; kDw divides each group's own stages)
  int out_type;
  bool big;      // kFwd, kDx: the weights in use are more than kStreamMin bytes
};

constexpr int kMaxSplits = 16;
constexpr size_t kPartMax = (size_t)64 << 20;  // partial sums of a split reduction, at most
constexpr int kCus = 256;
// Weights larger than this are taken not to stay in the 256 MB memory-side cache
// until their next use.  (Measured with calls on the same weights one after the
// other; a program that runs other layers in between finds smaller ones cold too.)
constexpr size_t kStreamMin = (size_t)100 << 20;

// Block shapes and their costs (us, but for the factor of a product's kind
// below): a stage of a block that has its compute unit to itself on a half-empty
// card (`alone`), a stage per compute unit with every one full (`full`), and a
// block's start and end (`edge`).  These and the constants of choose() are
// fitted to the times of every shape and split on 1040 products (260 random
// sizes, 1 to 8192 rows, 1 to 48 groups, widths 64 to 8192); fp8's two factors
// were set by hand (1.8 % from the best on average; the fit's, 1.24 and 1.39: 1.7).
struct Cost {
  int ta, tb, occ;
  float alone, full, edge;
};
constexpr int kShapes = 7;
constexpr Cost kCost[kShapes] = {
    {256, 256, 1, 1.25f, 1.39f, 6.6f},    // most arithmetic per byte moved: large products
    {256, 128, 1, 0.75f, 0.855f, 4.3f},   // groups of about 100 rows: the weights pass through LDS once
    {128, 128, 2, 0.77f, 0.785f, 3.5f},   // two blocks a compute unit: one stores while the other computes
    {128, 64, 2, 0.63f, 0.38f, 2.9f},     // fewer rows a group
    {128, 64, 1, 0.30f, 0.43f, 2.6f},     // the same by two teams: few tiles, a long reduction
    {128, 32, 2, 0.285f, 0.415f, 1.6f},  // decode: the stream of the weights
    {256, 192, 1, 1.00f, 1.19f, 5.3f},    // where 256 x 256 leaves compute units idle in its last round
};
// Factors of `alone` and `full`: 16-bit forward, dx, dw, fp8 forward.
constexpr float kAlone[4] = {0.99f, 0.80f, 0.92f, 1.15f};
constexpr float kFull[4] = {1.09f, 0.80f, 0.39f, 1.12f};

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct Choice {
  int shape;
  Plan plan;
};

// The shape and the number of splits with the smallest estimate of
//   max(rounds of blocks in sequence, the work at the full card's rate, the
//   staged bytes at 14.8 TB/s) + the join of the splits.
// The groups' sizes are on the device; the estimate takes them as equal, with
// half a tile of waste each, and all of `rows` as in use.  On 1256 products the
// choice is 2.0 % from the best on average, 6.8 % at the 90th percentile, 29 % at
// the 99th and 66 % at worst (dw of 1667 rows, 24 groups, 2024 x 256: 22 us for
// 13): nothing here counts the bytes past L2.  Where `rows` is a capacity of
// eight times the rows in groups, it is 31 % from the best on average (485 forward
// and dx products by group), 86 % at the 90th percentile.
inline Choice choose(int op, int in_type, int rows, int N, int K, int groups) {
  const int re = in_type == kFP8 ? 128 : 64;
  const int cols = op == kFwd ? N : K;
  const int live = op == kDw ? groups : (rows < groups ? rows : groups);  // groups with rows, at most
  const int nst = ceil_div(op == kFwd ? K : (op == kDx ? N : ceil_div(rows, groups)), re);
  const int kind = in_type == kFP8 ? 3 : op;
  const float alone = kAlone[kind], full = kFull[kind];
  const float out = (op == kDw ? (float)groups * N : (float)rows) * ((cols + 3) & ~3);
  Choice best{};
  float best_us = 0.0f;
  for (int s = 0; s < kShapes; ++s) {
    const Cost& c = kCost[s];
    if (op == kDw && (c.tb & (c.tb - 1))) continue;  // its rows are read transposed: powers of two
    const int nca = ceil_div(cols, c.ta);
    int nrb;      // row tiles a group (kDw) or at most in all
    float tiles;  // expected in all
    if (op == kDw) {
      nrb = ceil_div(N, c.tb);
      tiles = (float)nrb * nca * groups;
    } else {
      nrb = rows / c.tb + live;
      const float part = live ? (float)rows / live / c.tb : 0.0f;
      const float each = groups == 1 ? ceilf(part) : 0.5f * (part + 0.5f + ceilf(part));
      tiles = (each > 1.0f ? each : 1.0f) * live * nca;
    }
    static constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, kMaxSplits};
    for (const int want : kSplits) {
      if (want > 1 && (tiles * want > 4 * kCus || want * 4 > nst || out * 4 * want > (float)kPartMax)) break;
      const int sps = ceil_div(nst > 0 ? nst : 1, want);
      const int splits = op == kDw ? want : ceil_div(nst > 0 ? nst : 1, sps);
      const float blocks = tiles * splits, rounds = ceilf(blocks / (kCus * c.occ));
      const float seq = rounds * (sps * c.alone * alone + c.edge);
      const float work = blocks / kCus * sps * c.full * full + c.edge;
      const float bytes = blocks * sps * (float)(c.ta + c.tb) * 128.0f / 14.8e6f;
      float us = seq > work ? seq : work;
      us = us > bytes ? us : bytes;
      if (splits > 1) us += 2.9f + splits * (0.17f + out * 8 / 6.5e6f);
      if (best_us == 0.0f || us < best_us) {
        best_us = us;
        best.shape = s;
        best.plan.nca = nca;
        best.plan.nrb = nrb;
        best.plan.splits = splits;
        best.plan.sps = sps;
      }
    }
  }
  return best;
}

// The forward product of a few rows in all takes k_linear_few while the blocks
// of groups with rows are no more than the compute units, and those of groups
// without few enough to come and go (measured: one row, 4096 x 7168: 7.9 us
// against 10.4 by tiles; 9 rows of 11 groups, 1140 x 752, up to 648 live blocks:
// 12.3 us against 7.6).
inline bool few_rows(int rows, int N, int groups) {
  const long each = ceil_div(N, 16), live = rows < groups ? rows : groups;
  return rows <= 16 && live * each <= kCus && groups * each <= 8 * kCus;
}

// Partial sums of any split that choose() may take for this product.
inline size_t part_bytes(int op, int rows, int N, int K, int groups) {
  const int cols = op == kFwd ? N : K;
  const size_t one = (op == kDw ? (size_t)groups * N : (size_t)rows) * ((cols + 3) & ~3) * sizeof(float);
  if (2 * one > kPartMax) return 0;
  return one * kMaxSplits < kPartMax ? one * kMaxSplits : kPartMax;
}

// Whether the weights in use pass the caches (`Plan::big`).
inline bool streams(int in_type, int rows, int N, int K, int groups) {
  return (size_t)(rows < groups ? rows : groups) * N * K * (in_type == kFP8 ? 1 : 2) > kStreamMin;
}

}  // namespace moe
