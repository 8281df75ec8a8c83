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
// An operand whose reduction is not contiguous is read from LDS with the
// transposing load.  fp8: the scales of a 128-column stage are constant over it, so
// one 16x16x128 product per tile is scaled by xs * ws in f32 and added to an
// f32 accumulator.
//
// Bound by the staging into LDS nearly everywhere (us, and with the products
// left out): fp8 8192 x 4096 x 7168 207 (2.3 PFLOP/s) and 182; 48 fp8 experts at
// 6144 rows 191 and 183; 48 bf16 experts 630 and 630 (5 TB/s past L2); 512 fp8
// rows 23 and 21.  With few rows an expert the weights stream at 6.9 TB/s.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_internal.hpp"
#include "linear_plan.hpp"
#include "moe_device.hpp"

namespace moe {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kXcd = 8;  // accelerator dies; block b runs on die b % 8, each has its own L2

// LDS pointers.  The DMA target and the tiles being read are passed to one
// inlined function as __restrict__: the compiler then knows that a read does
// not depend on the DMA in flight and places no wait between them.
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) v4i lds_v4i;
typedef __attribute__((address_space(3))) float lds_f32;
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) void* lds_void;

template <int AUX>
using Hint = std::integral_constant<int, AUX>;  // cache policy bits of a load: 2 = read once

constexpr uint32_t kOob = 0x80000000u;  // a buffer offset past every buffer used here: the load gives zeros

template <int IN>
__device__ __forceinline__ v4f mfma16(v4i a, v4i b, v4f c) {  // 16x16x32, 16-bit types
  if constexpr (IN == kBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// 16x16x128 of e4m3 operands, no block scales.  The instruction takes 32
// products at a time, aligns them to the largest and keeps about 14 bits below its
// leading one: the one place where a sum has fewer bits than f32's.  It is the
// price of the fp8 rate (an exact product of two e4m3 blocks would go through the
// 16-bit instructions, at half of it), and it leaves outputs in bf16 as far from
// the 64-bit values as f32 sums do (0.0017 normwise both, reductions of 2048 and
// 7168 columns).
__device__ __forceinline__ v4f mfma8(v8i a, v8i b, v4f c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, kFmtFp8, kFmtFp8, 0, 0, 0, 0);
}

// A 16-byte store at any multiple of the output type's size (rows of an odd
// number of 16-bit values start at odd multiples of 2 bytes).
typedef v4i v4i_any __attribute__((aligned(2)));
__device__ __forceinline__ void store16(void* p, v4i v) { *static_cast<v4i_any*>(p) = v; }

// Rows [lo, hi) of group g.  Offsets outside [0, rows], or falling, break the
// caller's contract; they are clamped so that no row outside the tensors is
// touched.
__device__ __forceinline__ void group_rows(const int32_t* off, int g, int rows, int& lo, int& hi) {
  lo = off ? min(max(off[g], 0), rows) : 0;
  hi = off ? min(max(off[g + 1], lo), rows) : rows;
}

// Row tiles of TB rows, counted over the groups in order.  Every wave does this
// by itself: 64 groups at a time, one per lane, prefix sums across the lanes.
// The first 64 groups' rows stay in registers, so that up to 64 groups cost one
// trip to memory in all (three dependent ones, for the count, the search and the
// group's rows, took 0.5 us longer).
template <int TB>
struct RowTiles {
  const int32_t* off;
  int groups, rows;
  int lo, hi, incl;  // of group `lane`: its rows, and the tiles up to its end
  int total;         // row tiles of all groups

  __device__ __forceinline__ int load(int c, int base, int& lo_, int& hi_) const {  // of groups [c, c + 64)
    const int lane = threadIdx.x & 63;
    lo_ = hi_ = 0;
    if (c + lane < groups) group_rows(off, c + lane, rows, lo_, hi_);
    int n = (hi_ - lo_ + TB - 1) / TB;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int up = __shfl_up(n, d);
      if (lane >= d) n += up;
    }
    return n + base;
  }
  __device__ __forceinline__ RowTiles(const int32_t* off_, int groups_, int rows_) : off(off_), groups(groups_), rows(rows_) {
    incl = load(0, 0, lo, hi);
    total = __builtin_amdgcn_readlane(incl, 63);
    for (int c = 64; c < groups; c += 64) {
      int l, h;
      total = __builtin_amdgcn_readlane(load(c, total, l, h), 63);
    }
  }
  // The group g of row tile `tile` < total, the tile's index t there, and the group's rows.
  __device__ __forceinline__ void find(int tile, int& g, int& t, int& glo, int& ghi) const {
    int c = 0, l = lo, h = hi, n = incl;
    unsigned long long past = __ballot(n > tile);
    while (!past && c + 64 < groups) {
      c += 64;
      n = load(c, __builtin_amdgcn_readlane(n, 63), l, h);
      past = __ballot(n > tile);
    }
    const int k = past ? __ffsll(past) - 1 : 63;  // tile < total: there is one
    g = c + k;
    glo = __builtin_amdgcn_readlane(l, k);
    ghi = __builtin_amdgcn_readlane(h, k);
    t = tile - (__builtin_amdgcn_readlane(n, k) - (ghi - glo + TB - 1) / TB);
  }
};

// Shape of a block's work.  TA x TB: columns x rows of its output tile; WA x WB
// waves; KS: teams of that many waves, each with its own LDS ring and every
// KS-th stage; NS: stages of a ring; OCC: blocks per compute unit the
// registers must allow.
template <int IN_, int OP_, int TA_, int TB_, int WA_, int WB_, int KS_, int NS_, int OCC_>
struct Shape {
  static constexpr int IN = IN_, OP = OP_, TA = TA_, TB = TB_, WA = WA_, WB = WB_, KS = KS_, NS = NS_, OCC = OCC_;
  static constexpr int W = WA * WB;
  static constexpr int ES = IN == kFP8 ? 1 : 2;
  static constexpr int RE = 128 / ES;               // reduction elements per stage
  static constexpr bool AT = OP != kFwd;            // operand stored with its columns contiguous (read transposed)
  static constexpr bool BT = OP == kDw;
  static constexpr int TI = TA / WA / 16, TJ = TB / WB / 16;  // 16 x 16 tiles per wave
  static constexpr int NA = TA / 8 / W, NB = TB / 8 / W;      // 1 KB DMA instructions per wave and stage
  static constexpr int NI = NA + NB;
  static constexpr int kSlot = (TA + TB) * 128;
  // fp8 scales: two buffers of four stages' values: 16 bytes a row, then 16
  // bytes per 128 columns (written by whole waves)
  static constexpr int kRowSc = (TB < 64 ? 64 : TB) * 16;
  static constexpr int kScale = IN == kFP8 ? kRowSc + 1024 : 0;
  static constexpr int kTeam = NS * kSlot + 2 * kScale;  // LDS of a team
  static constexpr int PRE = NS - 1;
  static constexpr int U = IN == kFP8 ? TI : 2 * TI;  // steps of a stage (below)
  static constexpr int D = IN == kFP8 ? 2 : 3;        // steps that operands are read ahead
  static constexpr int P = NS == 2 ? U / 2 : U;       // steps that the next DMA is issued in
  static constexpr int kLag = TJ == 1 ? 2 : 3;
  static_assert(U % 4 == 0 && D < 4 && kLag < 4 && (IN != kFP8 || kLag <= (U - D) * TJ), "rings of four");
  static_assert(NA * W * 8 == TA && NB * W * 8 == TB && TI * WA * 16 == TA && TJ * WB * 16 == TB, "tile shape");
  static_assert((!AT || (TA & (TA - 1)) == 0) && (!BT || (TB & (TB - 1)) == 0), "transposed rows are permuted in powers of two");
  static_assert(PRE * NI + 1 < 64, "vmcnt range");
  static_assert(IN != kFP8 || TB / 64 < W, "a wave for the weight scales");
  static_assert(KS * kTeam <= 160 * 1024, "LDS");
  static_assert(KS == 1 || TA * TB * 4 <= NS * kSlot, "a team's sums fit its ring");
  static_assert(KS == 1 || KS == 2, "teams share groups of four stages");
};

template <class C>
__global__ void __launch_bounds__(C::KS * C::W * 64, C::OCC * C::KS * C::W / 4) k_linear(LinearArgs p, Plan pl) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the kernel's name alone, and not every device builtin type-checks there
  constexpr int TA = C::TA, TB = C::TB, TI = C::TI, TJ = C::TJ, W = C::W, ES = C::ES, NS = C::NS, PRE = C::PRE;
  constexpr int IN = C::IN, OP = C::OP;
  __shared__ __align__(1024) uint8_t ring[C::KS * C::kTeam];
  const int tid = threadIdx.x, lane = tid & 63;
  const int team = __builtin_amdgcn_readfirstlane(tid >> 6) / W, wave = __builtin_amdgcn_readfirstlane(tid >> 6) % W;
  const int l16 = lane & 15, q = lane >> 4;
  const int wa = wave % C::WA, wb = wave / C::WA;
  const int cols = OP == kFwd ? p.N : p.K;

  // ---- the block's tile.  Consecutive items share an XCD: inside a group,
  // bands of four column tiles, row by row, so that the 32 tiles a die works
  // on at one time read about 4 column and 8 row operands.
  int g, lo, hi, c0, r0, nr, nred, split;
  size_t row0;  // the tile's first row in the output
  // Weights that leave the caches before they are needed again are loaded with
  // the streaming policy (measured, us: 48 fp8 experts at 8 rows 233 -> 204, 48
  // bf16 experts at 6144 uneven rows 645 -> 631; dx of 4 experts of 7168 x 2048
  // at 4096 rows 163 -> 153).  Not where many row tiles share them (one expert
  // of 8192 x 8192: dx 782 -> 799; forward with two row tiles sharing: 662 for
  // the 645 above), nor where they stay in the memory-side cache (77 x 2041 x
  // 7152 in fp8: 12.7 -> 16.5).
  bool once = false;
  {
    const int xcd = blockIdx.x % kXcd, j = blockIdx.x / kXcd;
    if (OP == kDw) {
      // every die takes its share of each group, so that uneven groups spread
      const int per = pl.nca * pl.nrb, share = (per * pl.splits + kXcd - 1) / kXcd;
      g = j / share;
      int l = xcd * share + j % share;
      if (l >= per * pl.splits) return;
      split = l / per;
      l -= split * per;
      group_rows(p.off, g, p.rows, lo, hi);
      const int band = l / (pl.nrb * 4), rem = l - band * pl.nrb * 4, w = min(4, pl.nca - 4 * band);
      r0 = rem / w * TB;
      c0 = (4 * band + rem % w) * TA;
      nr = min(TB, p.N - r0);
      nred = hi - lo;
      row0 = (size_t)g * p.N + r0;
    } else {
      const RowTiles<TB> rt(p.off, p.groups, p.rows);
      const int tiles = rt.total * pl.nca;
      const int items = tiles * pl.splits, share = (items + kXcd - 1) / kXcd;
      const int item = xcd * share + j;
      if (j >= share || item >= items) return;
      split = item / tiles;
      const int l0 = item - split * tiles;
      int t;
      rt.find(l0 / pl.nca, g, t, lo, hi);
      const int nrb = (hi - lo + TB - 1) / TB, l = t * pl.nca + l0 % pl.nca;
      const int band = l / (nrb * 4), rem = l - band * nrb * 4, w = min(4, pl.nca - 4 * band);
      r0 = lo + rem / w * TB;
      c0 = (4 * band + rem % w) * TA;
      nr = min(TB, hi - r0);
      once = pl.big && nrb <= (OP == kDx ? 8 : 1);
      nred = OP == kFwd ? p.K : p.N;
      row0 = (size_t)r0;
    }
  }
  const int nst = (nred + C::RE - 1) / C::RE;
  int s_lo, s_n;  // the block's stages; its teams take them in turn
  {
    const int sps = OP == kDw ? (nst + pl.splits - 1) / pl.splits : pl.sps;
    s_lo = min(nst, split * sps);
    s_n = min(sps, nst - s_lo);
  }

  // ---- DMA.  A contiguous-reduction operand is staged as rows of 128 bytes,
  // 8 rows per instruction; a transposed one as reduction rows of T columns.
  // The 16-byte pieces of a row are permuted so that the reads below spread
  // over the LDS banks.
  const int ldr = OP == kFwd ? p.K : p.N;  // row length of a contiguous-reduction operand
  const uint8_t *abase, *bbase;
  uint32_t alim = 0, blim = 0;
  const uint8_t* wslab = static_cast<const uint8_t*>(p.a) + (OP == kDw ? 0 : (size_t)g * p.N * p.K * ES);
  if (OP == kFwd) {
    abase = wslab + (size_t)c0 * p.K * ES;
    alim = (uint32_t)min(TA, p.N - c0) * (uint32_t)(p.K * ES);
  } else if (OP == kDx) {
    abase = wslab + (size_t)c0 * 2;
  } else {
    abase = static_cast<const uint8_t*>(p.a) + ((size_t)lo * p.K + c0) * 2;
  }
  if (OP == kDw) {
    bbase = static_cast<const uint8_t*>(p.b) + ((size_t)lo * p.N + r0) * 2;
  } else {
    bbase = static_cast<const uint8_t*>(p.b) + (size_t)r0 * ldr * ES;
    blim = (uint32_t)nr * (uint32_t)(ldr * ES);
  }
  // Lane offsets of an operand's first instruction; instruction m is a uniform
  // distance further.  (Rows 32 apart permute their pieces alike.)
  auto kc_row = [&]() { return 8 * wave + (lane >> 3); };
  auto kc_piece = [&]() { return (lane & 7) ^ (kc_row() & 7); };
  auto mc_off = [&](int T, int ld, int ncol) {
    const int PR = T / 8, RPI = 64 / PR;  // pieces per row, rows per instruction
    const int row = wave * RPI + lane / PR;
    const int f = (row & 3) | ((row >> 1) & 4);
    const int pc = (lane % PR) ^ ((2 * f) & (PR - 1));
    return 8 * pc < ncol ? ((uint32_t)row * (uint32_t)ld + 8u * pc) * 2u : kOob;
  };
  const uint32_t kpc = 16u * (uint32_t)kc_piece();
  const uint32_t rowb = (uint32_t)(ldr * ES);
  const uint32_t avo = C::AT ? mc_off(TA, p.K, cols - c0) : (uint32_t)kc_row() * rowb + kpc;
  const uint32_t bvo = C::BT ? mc_off(TB, p.N, nr) : (uint32_t)kc_row() * rowb + kpc;
  const uint32_t astep = C::AT ? (uint32_t)(W * (512 / TA) * p.K * 2) : 8 * W * rowb;
  const uint32_t bstep = C::BT ? (uint32_t)(W * (512 / TB) * p.N * 2) : 8 * W * rowb;

  // fp8 scales, four stages at a time, 16 bytes a lane: waves [0, TB / 64) load
  // the rows', the last wave the weights' of each 128 columns of the tile.
  // (A dword a row and stage, 64 lines an instruction, kept the address unit
  // busy: 8192 x 4096 x 7168 took 8 % longer.)
  const int nkb = (p.K + 127) / 128, nnb = (p.N + 127) / 128;
  const float* scp = nullptr;
  uint32_t sclim = 0, scvo = kOob;
  const bool scw = IN == kFP8 && (wave < (TB + 63) / 64 || wave == W - 1);
  if constexpr (IN == kFP8) {
    if (wave < (TB + 63) / 64) {
      scp = p.bs + (size_t)r0 * nkb;
      sclim = (uint32_t)(nr * nkb) * 4u;
      if (wave * 64 + lane < TB) scvo = (uint32_t)((wave * 64 + lane) * nkb) * 4u;
    } else if (wave == W - 1) {
      scp = p.as + ((size_t)g * nnb + c0 / 128) * nkb;
      sclim = (uint32_t)((nnb - c0 / 128) * nkb) * 4u;
      if (lane < (TA + 127) / 128) scvo = (uint32_t)(lane * nkb) * 4u;
    }
    // wave-uniform by construction; said so, for the buffer descriptor
    const uint64_t a = (uint64_t)(uintptr_t)scp;
    scp = reinterpret_cast<const float*>((uintptr_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32 |
                                                     (uint32_t)__builtin_amdgcn_readfirstlane((int)a)));
    sclim = (uint32_t)__builtin_amdgcn_readfirstlane((int)sclim);
  }
  auto dma_scales = [&](lds_u8* dst, int st) __attribute__((always_inline)) {  // of stages st .. st + 3
    // the stage goes into the checked offset: a row's last four may end past it
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(scp, sclim),
                                             (lds_void)(dst + (wave == W - 1 ? C::kRowSc : wave * 1024)), 16,
                                             scvo + (uint32_t)st * 4u, 0, 0, 0);
  };

  // DMA instruction m of stage st into a ring slot.  Stages past the end load
  // nothing (their buffers have no bytes), so that every stage counts the
  // same number of loads.
  auto dma = [&](auto aux, lds_u8* wr, int st, int m, bool live) __attribute__((always_inline)) {
    auto kc = [&](auto hint, const uint8_t* base, uint32_t lim, uint32_t vo, uint32_t step, int m, lds_u8* dst) {
      const uint32_t so = (uint32_t)st * 128u;
      const uint32_t v = so + kpc < rowb ? vo : kOob;  // pieces past the row's end
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(base, live ? lim : 0u), (lds_void)(dst + (wave + W * m) * 1024), 16,
                                               v + (uint32_t)m * step, so, 0, decltype(hint)::value);
    };
    auto mc = [&](auto hint, const uint8_t* base, int ld, int col0, uint32_t vo, uint32_t step, int m, lds_u8* dst) {
      const int rows = live ? min(C::RE, nred - st * C::RE) : 0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          make_rsrc(base + (size_t)st * C::RE * ld * 2, rows > 0 ? (uint32_t)(rows * ld - col0) * 2u : 0u),
          (lds_void)(dst + (wave + W * m) * 1024), 16, vo + (uint32_t)m * step, 0, 0, decltype(hint)::value);
    };
    if (m < C::NA) {
      if (C::AT) mc(aux, abase, p.K, c0, avo, astep, m, wr);
      else kc(aux, abase, alim, avo, astep, m, wr);
    } else if (m < C::NA + C::NB) {
      if (C::BT) mc(Hint<0>{}, bbase, p.N, r0, bvo, bstep, m - C::NA, wr + TA * 128);
      else kc(Hint<0>{}, bbase, blim, bvo, bstep, m - C::NA, wr + TA * 128);
    }
  };

  // ---- LDS reads.  Contiguous reduction: lane (l16, q) of a tile reads pieces
  // q and q + 4 of its row.  Transposed: a 16-lane group reads four reduction
  // rows of 16 columns, each lane getting one column's four values.
  const int fa = C::AT ? (l16 >> 2) | ((q & 1) << 2) : l16 & 7;
  const int fb = C::BT ? (l16 >> 2) | ((q & 1) << 2) : l16 & 7;
  const uint32_t ra = (uint32_t)(wa * TI * 16 + l16) * 128;
  const uint32_t rb = (uint32_t)(TA * 128 + (wb * TJ * 16 + l16) * 128);
  auto ld_kc = [&](const lds_u8* rd, uint32_t row, int kk, int f) {
    return *reinterpret_cast<const lds_v4i*>(rd + row + (((4 * kk + q) ^ f) * 16));
  };
  auto ld_mc = [&](const lds_u8* rd, int T, int tile, int kk, int f) {
    const int row = 32 * kk + 8 * q + (l16 >> 2);
    const lds_u8* a = rd + row * T * 2 + (((tile ^ f) & (T / 16 - 1)) | (tile & ~(T / 16 - 1))) * 32 + (l16 & 3) * 8;
    const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)a);
    const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(a + 4 * T * 2));
    typedef short v8s __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(v4i, (v8s)__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto lda = [&](const lds_u8* rd, int i, int kk) {
    if constexpr (C::AT) return ld_mc(rd, TA, wa * TI + i, kk, fa);
    else return ld_kc(rd, ra + (uint32_t)(i * 16) * 128, kk, fa);
  };
  auto ldb = [&](const lds_u8* rd, int j, int kk) {
    if constexpr (C::BT) return ld_mc(rd + TA * 128, TB, wb * TJ + j, kk, fb);
    else return ld_kc(rd, rb + (uint32_t)(j * 16) * 128, kk, fb);
  };

  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // ---- main loop.  A stage is U steps of one A tile against all of the wave's
  // B tiles (fp8: whole 128 columns; 16-bit: half by half).  A's operands are
  // read D steps ahead, and the last D steps of a stage run after the barrier
  // that ends it, from registers, while the next stage's first operands are on
  // their way: no wave stands at the start of a stage waiting for LDS.  The
  // next DMA is issued in between, instruction by instruction: over the whole
  // stage in a deeper ring, over its first half in one of two stages, where it
  // has to land by the stage's end (bf16 8192^3: 869 us over all of it, 799
  // over half, 802 over a quarter).  fp8: a tile's
  // product is scaled and added kLag products later, when it is long finished.
  constexpr int U = C::U, D = C::D, kLag = C::kLag;
  constexpr int KH = U / TI;  // halves of a stage
  v8i a[IN == kFP8 ? 4 : 1], b[IN == kFP8 ? TJ : 1];
  v4i ah[IN == kFP8 ? 1 : 4], bh[IN == kFP8 ? 1 : 2][TJ];
  float sold[TJ], snew[TJ], wsc = 0.f;
  v4f part[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (IN == kFP8) a[i] = v8i{0, 0, 0, 0, 0, 0, 0, 0};
    else ah[i] = v4i{0, 0, 0, 0};
  }
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    sold[j] = snew[j] = 0.f;
    if constexpr (IN == kFP8) b[j] = v8i{0, 0, 0, 0, 0, 0, 0, 0};
    else bh[0][j] = bh[1][j] = v4i{0, 0, 0, 0};
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[i] = v4f{0.f, 0.f, 0.f, 0.f};

  auto join8 = [](v4i x, v4i y) -> v8i { return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7); };
  auto read_a = [&](const lds_u8* rd, int u) __attribute__((always_inline)) {
    if constexpr (IN == kFP8) a[u % 4] = join8(lda(rd, u, 0), lda(rd, u, 1));
    else ah[u % 4] = lda(rd, u % TI, u / TI);
  };
  // fp8: adds product n (counted through the stage; negative: of the stage before)
  auto promote = [&](int n) __attribute__((always_inline)) {
    const int i = ((n + U * TJ) / TJ) % U, j = (n + U * TJ) % TJ;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc[i][j][e] = fmaf(part[(n + 4) % 4][e], n + kLag >= (U - D) * TJ || n < 0 ? sold[j] : snew[j], acc[i][j][e]);
  };
  auto step = [&](int u, const lds_u8* rd, bool read_next) __attribute__((always_inline)) {
    // reads for the steps ahead (rd: this stage for u < U - D, else the next)
    if (read_next) read_a(rd, (u + D) % U);
    if constexpr (IN == kFP8) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        part[(u * TJ + j) % 4] = mfma8(a[u % 4], b[j], v4f{0.f, 0.f, 0.f, 0.f});
        promote(u * TJ + j - kLag);
        if (read_next && u == U - 1) b[j] = join8(ldb(rd, j, 0), ldb(rd, j, 1));
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      if (read_next) {
#pragma unroll
        for (int h = 0; h < KH; ++h)
#pragma unroll
          for (int j = 0; j < TJ; ++j)  // B's next half, spread over the D steps before it
            if ((u + D - (j * D) / TJ) % U == h * TI) bh[h][j] = ldb(rd, j, h);
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[u % TI][j] = mfma16<IN>(ah[u % 4], bh[u / TI][j], acc[u % TI][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // From one barrier to the next: stage s's slot rd is complete, wr is free.
  // (swr, srd: the scales' buffers of the next and this group of four stages.)
  constexpr int kGroup = 4 / C::KS;  // this team's stages of a group
  auto body = [&](auto aux, lds_u8* __restrict__ wr, const lds_u8* __restrict__ rd, lds_u8* __restrict__ swr,
                  const lds_u8* __restrict__ srd, int s) __attribute__((always_inline)) {
    const int k = (s + PRE) * C::KS + team, st = s_lo + k;
    const bool live = k < s_n;
    if constexpr (IN == kFP8)  // before the stage's tiles, with which they are waited for
      if (scw && (s < 0 ? s == -PRE : s % kGroup == 0)) dma_scales(swr, s_lo + (s < 0 ? 0 : (s / kGroup + 1) * 4));
    if (s < 0) {
#pragma unroll
      for (int m = 0; m < C::NI; ++m) dma(aux, wr, st, m, live);
      return;
    }
#pragma unroll
    for (int v = 0; v < U; ++v) {
#pragma unroll
      for (int m = 0; m < C::NI; ++m)
        if (m * C::P / C::NI == v) dma(aux, wr, st, m, live);
      if constexpr (IN == kFP8) {
        if (v == 0) {
          const lds_f32* sc = reinterpret_cast<const lds_f32*>(srd) + ((s * C::KS + team) & 3);
          wsc = sc[C::kRowSc / 4 + 4 * ((wa * TI * 16) / 128)];
#pragma unroll
          for (int j = 0; j < TJ; ++j) {
            sold[j] = snew[j];
            snew[j] = sc[4 * (wb * TJ * 16 + 16 * j + l16)];
          }
          // the second team's stage past the end (all zeros) finds the next
          // row's scales, which may be NaN
          if (C::KS > 1 && s * C::KS + team >= s_n) {
            wsc = 0.f;
#pragma unroll
            for (int j = 0; j < TJ; ++j) snew[j] = 0.f;
          }
        }
        if (v == D) {
#pragma unroll
          for (int j = 0; j < TJ; ++j) snew[j] *= wsc;
        }
      }
      step((v + U - D) % U, rd, true);
    }
  };
  lds_u8* const ring0 = (lds_u8*)ring + team * C::kTeam;
  lds_u8* const scale0 = ring0 + NS * C::kSlot;
  const int steps = (s_n + C::KS - 1) / C::KS;
  auto run = [&](auto aux) __attribute__((always_inline)) {
    int wslot = 0, rslot = 0;
    for (int s = -PRE; s < steps; ++s) {
      if (s >= 0) {
        // this wave's part of stage s has landed (PRE - 1 younger stages may be
        // in flight) and its reads of stage s - 1 are done; then the barrier
        // says the same of every wave
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"((PRE - 1) * C::NI) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      const int par = s < 0 ? 1 : (s / kGroup) & 1;  // the prologue's group goes into buffer 0
      body(aux, ring0 + wslot * C::kSlot, ring0 + rslot * C::kSlot, scale0 + (par ^ 1) * C::kScale, scale0 + par * C::kScale, s);
      wslot = wslot == NS - 1 ? 0 : wslot + 1;
      if (s >= 0) rslot = rslot == NS - 1 ? 0 : rslot + 1;
    }
  };
  if (OP != kDw && once) run(Hint<2>{});
  else run(Hint<0>{});
  // the last stage's last steps
#pragma unroll
  for (int j = 0; j < TJ; ++j) sold[j] = snew[j];
#pragma unroll
  for (int u = U - D; u < U; ++u) step(u, nullptr, false);
  if constexpr (IN == kFP8) {
#pragma unroll
    for (int n = U * TJ - kLag; n < U * TJ; ++n) promote(n);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the block
  if constexpr (C::KS > 1) {
    // the teams' sums, added in order by the first
    __syncthreads();
    lds_f32* const sums = reinterpret_cast<lds_f32*>((lds_u8*)ring);
    typedef __attribute__((address_space(3))) v4f lds_v4f;
    auto at = [&](int t, int i, int j) {
      return reinterpret_cast<lds_v4f*>(sums + t * (C::kTeam / 4) + (((wave * TI + i) * TJ + j) * 64 + lane) * 4);
    };
    if (team > 0) {
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) *at(team, i, j) = acc[i][j];
    }
    __syncthreads();
    if (team > 0) return;
#pragma unroll
    for (int t = 1; t < C::KS; ++t)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] += *at(t, i, j);
  }

  // ---- the tile's values, rounded once to the output type.  Each wave turns
  // its 16-row strips in LDS (its share of the ring, two strips in turn where they fit), so
  // that a store writes whole rows of the wave's columns.  (A lane's own 4 to
  // 16 consecutive columns stored directly: 8192 x 4096 x 7168 in fp8 215 us
  // against 205, the weight gradients of 4 experts of 7168 x 2048 157 against 128.)
  __syncthreads();
  constexpr int CW = TI * 16;               // the wave's columns
  constexpr int kStrip = 16 * CW * 4;
  constexpr int kStrips = 2 * kStrip * W <= NS * C::kSlot ? 2 : 1;
  static_assert(kStrips * kStrip * W <= NS * C::kSlot, "strips fit the ring");
  typedef __attribute__((address_space(3))) v4f lds_v4f;
  lds_u8* const strip0 = (lds_u8*)ring + wave * kStrips * kStrip;
  auto write = [&](auto outc, void* out, int pitch) {
    constexpr int OUT = decltype(outc)::value;
    using O = std::conditional_t<OUT == kBF16, __bf16, std::conditional_t<OUT == kF16, _Float16, float>>;
    constexpr int V = 16 / sizeof(O);       // columns of a 16-byte store
    constexpr int LR = CW / V, RI = 64 / LR;  // lanes a row, rows an instruction
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      lds_u8* const strip = strip0 + j % kStrips * kStrip;
      // 16-byte chunk c of row r lies at chunk c ^ r: no two rows on one bank
#pragma unroll
      for (int i = 0; i < TI; ++i)
        *reinterpret_cast<lds_v4f*>(strip + l16 * CW * 4 + ((4 * i + q) ^ l16) * 16) = acc[i][j];
#pragma unroll
      for (int k = 0; k < 16 / RI; ++k) {
        const int rr = k * RI + lane / LR, c = (lane % LR) * V;
        const int r = wb * TJ * 16 + 16 * j + rr, cc = wa * CW + c;
        O* o = static_cast<O*>(out) + (row0 + r) * pitch + c0 + cc;
        if (r < nr) {
          if (c0 + cc + V <= cols) {
            O v[V];
#pragma unroll
            for (int h = 0; h < V / 4; ++h) {
              const v4f x = *reinterpret_cast<const lds_v4f*>(strip + rr * CW * 4 + ((c / 4 + h) ^ rr) * 16);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[4 * h + e] = (O)x[e];
            }
            v4i w;
            __builtin_memcpy(&w, v, 16);
            store16(o, w);
          } else {
#pragma unroll 1
            for (int e = 0; c0 + cc + e < cols; ++e)
              o[e] = (O) * reinterpret_cast<const lds_f32*>(strip + rr * CW * 4 + (((c + e) / 4) ^ rr) * 16 + (e & 3) * 4);
          }
        }
      }
    }
  };
  if (pl.splits > 1 || pl.out_type == kF32) {
    // partial sums: rows padded to 16 bytes
    const int pitch = pl.splits > 1 ? (cols + 3) & ~3 : cols;
    const size_t total = (size_t)(OP == kDw ? (size_t)p.groups * p.N : (size_t)p.rows) * pitch;
    write(std::integral_constant<int, kF32>{}, pl.splits > 1 ? static_cast<float*>(p.part) + split * total : p.out, pitch);
  } else if (IN == kF16 || (IN == kFP8 && pl.out_type == kF16)) {
    write(std::integral_constant<int, kF16>{}, p.out, cols);
  } else {
    write(std::integral_constant<int, kBF16>{}, p.out, cols);
  }
#endif
}

// ---- few rows: y for at most 16 rows in all.  The weights are read once,
// straight into the MFMA's operand registers: a block takes 16 columns of a
// group, its eight waves every eighth 128-byte piece of the rows, each kChunk
// pieces ahead; the waves' sums are added in order through LDS.  One launch, no
// partial sums in memory, and columns / 16 blocks a group.
constexpr int kFewWaves = 8;
constexpr int kChunk = 4;

// NT: the weights with the streaming policy (one row, 4096 x 7168 in fp8, cached:
// 1.2 us longer with it than the 7.9 without).
template <int IN, bool NT>
__global__ void __launch_bounds__(kFewWaves * 64) k_linear_few(LinearArgs p, int out_type) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int ES = IN == kFP8 ? 1 : 2;
  __shared__ __align__(16) float red[kFewWaves][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int g = blockIdx.y, c0 = blockIdx.x * 16;
  int lo, hi;
  group_rows(p.off, g, p.rows, lo, hi);  // p.rows <= 16
  if (hi == lo) return;
  const int nr = hi - lo;
  const uint32_t rowb = (uint32_t)(p.K * ES);
  const int npc = (int)(rowb + 127) / 128;  // 128-byte pieces of a row
  const int nkb = (p.K + 127) / 128, nnb = (p.N + 127) / 128;
  const rsrc_t Ar = make_rsrc(static_cast<const uint8_t*>(p.a) + ((size_t)g * p.N + c0) * rowb,
                              (uint32_t)min(16, p.N - c0) * rowb);
  const rsrc_t Br = make_rsrc(static_cast<const uint8_t*>(p.b) + (size_t)lo * rowb, (uint32_t)nr * rowb);
  const rsrc_t Sr = make_rsrc(IN == kFP8 ? p.bs + (size_t)lo * nkb : nullptr, IN == kFP8 ? (uint32_t)(nr * nkb) * 4u : 0u);
  const rsrc_t Tr = make_rsrc(IN == kFP8 ? p.as + ((size_t)g * nnb + c0 / 128) * nkb : nullptr,
                              IN == kFP8 ? (uint32_t)nkb * 4u : 0u);
  v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
  struct Piece {
    v4i a[2], b[2];
    int xs, ws;
  };
  Piece buf[2][kChunk];
  // piece pc of the row: lane (l16, q) takes bytes [16 q, 16 q + 16) and the
  // same of its upper half; past the row's or the tensor's end, zeros
  auto fetch = [&](Piece& x, int pc) {
    const uint32_t o = (uint32_t)pc * 128u + 16u * q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = o + 64u * h < rowb ? (uint32_t)l16 * rowb + o + 64u * h : kOob;
      x.a[h] = buf_load16_p<NT ? 2 : 0>(Ar, at, 0);
      x.b[h] = buf_load16(Br, at, 0);
    }
    if constexpr (IN == kFP8) {
      x.ws = buf_load4(Tr, pc < nkb ? 4u * pc : kOob, 0);
      x.xs = buf_load4(Sr, pc < nkb ? (uint32_t)(l16 * nkb + pc) * 4u : kOob, 0);
    }
  };
  auto add = [&](const Piece& x) {
    if constexpr (IN == kFP8) {
      const float s = __int_as_float(x.xs) * __int_as_float(x.ws);
      const v8i a = __builtin_shufflevector(x.a[0], x.a[1], 0, 1, 2, 3, 4, 5, 6, 7);
      const v8i b = __builtin_shufflevector(x.b[0], x.b[1], 0, 1, 2, 3, 4, 5, 6, 7);
      const v4f d = mfma8(a, b, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(d[e], s, acc[e]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) acc = mfma16<IN>(x.a[h], x.b[h], acc);
    }
  };
#pragma unroll
  for (int k = 0; k < kChunk; ++k) fetch(buf[0][k], wave + kFewWaves * k);
  for (int p0 = wave; p0 < npc; p0 += 2 * kChunk * kFewWaves) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int base = p0 + h * kChunk * kFewWaves;
#pragma unroll
      for (int k = 0; k < kChunk; ++k) fetch(buf[h ^ 1][k], base + (kChunk + k) * kFewWaves);
#pragma unroll
      for (int k = 0; k < kChunk; ++k) add(buf[h][k]);
    }
  }
  *reinterpret_cast<v4f*>(&red[wave][l16 * 16 + 4 * q]) = acc;
  __syncthreads();
  const int r = tid >> 4, c = c0 + (tid & 15);
  if (r < nr && c < p.N) {
    float s = red[0][tid];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += red[w][tid];
    const size_t o = (size_t)(lo + r) * p.N + c;
    if (out_type == kF32) static_cast<float*>(p.out)[o] = s;
    else if (out_type == kF16) static_cast<_Float16*>(p.out)[o] = (_Float16)s;
    else static_cast<__bf16*>(p.out)[o] = (__bf16)s;
  }
#endif
}

// out = sum of the splits' partial sums, in split order, four columns a thread;
// four splits' loads are in flight at a time.  kFwd, kDx: rows in no group have
// no sums and are left alone.
template <int OUT>
__global__ void __launch_bounds__(256) k_linear_join(LinearArgs p, int rows, int cols, int splits, bool rows_out) {
  using O = std::conditional_t<OUT == kBF16, __bf16, std::conditional_t<OUT == kF16, _Float16, float>>;
  const uint32_t quads = (uint32_t)(cols + 3) / 4;
  const size_t total = (size_t)rows * quads;
  size_t i0 = 0, i1 = total;
  if (rows_out && p.off) {
    i0 = (size_t)min(max(p.off[0], 0), rows) * quads;
    i1 = (size_t)min(max(p.off[p.groups], 0), rows) * quads;
  }
  const v4f* part = static_cast<const v4f*>(p.part);
  for (size_t i = i0 + (size_t)blockIdx.x * 256 + threadIdx.x; i < i1; i += (size_t)gridDim.x * 256) {
    v4f s = part[i];
    for (int z = 1; z < splits; z += 4) {
      v4f x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = part[(size_t)min(z + k, splits - 1) * total + i];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (z + k < splits) s += x[k];
    }
    const size_t row = i / quads;
    const int c = (int)(i - row * quads) * 4;
    O* o = static_cast<O*>(p.out) + row * cols + c;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < cols) o[e] = (O)s[e];
  }
}

template <class C>
hipError_t run_shape(const LinearArgs& p, const Plan& pl, hipStream_t st) {
  long blocks;
  if (C::OP == kDw) blocks = (long)p.groups * (ceil_div(pl.nca * pl.nrb * pl.splits, kXcd) * kXcd);
  else blocks = (long)ceil_div(pl.nca * pl.nrb * pl.splits, kXcd) * kXcd;
  k_linear<C><<<dim3((unsigned)blocks), C::KS * C::W * 64, 0, st>>>(p, pl);
  return hipGetLastError();
}

template <int IN, int OP>
hipError_t run_op(int out_type, LinearArgs p, void* ws, hipStream_t st) {
  const bool big = streams(IN, p.rows, p.N, p.K, p.groups);
  if constexpr (OP == kFwd) {
    if (few_rows(p.rows, p.N, p.groups)) {
      const dim3 grid((unsigned)ceil_div(p.N, 16), p.groups);
      if (big) k_linear_few<IN, true><<<grid, kFewWaves * 64, 0, st>>>(p, out_type);
      else k_linear_few<IN, false><<<grid, kFewWaves * 64, 0, st>>>(p, out_type);
      return hipGetLastError();
    }
  }
  Choice c = choose(OP, IN, p.rows, p.N, p.K, p.groups);
  c.plan.out_type = out_type;
  c.plan.big = big;
  p.part = ws;
  hipError_t e;
  if (c.shape == 0) e = run_shape<Shape<IN, OP, 256, 256, 2, 4, 1, 2, 1>>(p, c.plan, st);
  else if (c.shape == 1) e = run_shape<Shape<IN, OP, 256, 128, 4, 2, 1, 3, 1>>(p, c.plan, st);
  else if (c.shape == 2) e = run_shape<Shape<IN, OP, 128, 128, 2, 2, 1, 2, 2>>(p, c.plan, st);
  else if (c.shape == 3) e = run_shape<Shape<IN, OP, 128, 64, 2, 2, 1, 3, 2>>(p, c.plan, st);
  else if (c.shape == 4) e = run_shape<Shape<IN, OP, 128, 64, 2, 2, 2, 3, 1>>(p, c.plan, st);
  else if (c.shape == 5) e = run_shape<Shape<IN, OP, 128, 32, 2, 2, 1, 3, 2>>(p, c.plan, st);
  else if constexpr (OP != kDw) e = run_shape<Shape<IN, OP, 256, 192, 2, 4, 1, 2, 1>>(p, c.plan, st);
  else return hipErrorInvalidValue;  // choose() does not take it for kDw
  if (e != hipSuccess || c.plan.splits == 1) return e;
  const int cols = OP == kFwd ? p.N : p.K;
  const int rows = OP == kDw ? p.groups * p.N : p.rows;  // a split output is at most kPartMax
  const size_t want = ((size_t)rows * ceil_div(cols, 4) + 255) / 256;
  const unsigned blocks = (unsigned)(want < 2048 ? want : 2048);
  if (out_type == kBF16) k_linear_join<kBF16><<<blocks, 256, 0, st>>>(p, rows, cols, c.plan.splits, OP != kDw);
  else if (out_type == kF16) k_linear_join<kF16><<<blocks, 256, 0, st>>>(p, rows, cols, c.plan.splits, OP != kDw);
  else k_linear_join<kF32><<<blocks, 256, 0, st>>>(p, rows, cols, c.plan.splits, OP != kDw);
  return hipGetLastError();
}

template <int IN>
hipError_t run_in(int op, int out_type, const LinearArgs& p, void* ws, hipStream_t st) {
  if (op == kFwd) return run_op<IN, kFwd>(out_type, p, ws, st);
  if (op == kDx) return run_op<IN, kDx>(out_type, p, ws, st);
  return run_op<IN, kDw>(out_type, p, ws, st);
}

}  // namespace

size_t linear_workspace(int rows, int N, int K, int groups, int in_type) {
  size_t n = part_bytes(kFwd, rows, N, K, groups);
  if (in_type != kFP8)
    for (int op = kDx; op <= kDw; ++op) {
      const size_t m = part_bytes(op, rows, N, K, groups);
      n = m > n ? m : n;
    }
  return n;
}

hipError_t launch_linear(int op, int in_type, int out_type, const LinearArgs& p, void* ws, hipStream_t st) {
  if (in_type == kFP8) return run_op<kFP8, kFwd>(out_type, p, ws, st);
  return in_type == kBF16 ? run_in<kBF16>(op, out_type, p, ws, st) : run_in<kF16>(op, out_type, p, ws, st);
}

}  // namespace moe
