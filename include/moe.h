/*
 * moe.h -- C ABI of libmoe: one MI355X's share of a fused Mixture-of-Experts
 * layer (sigmoid top-k routing, EPLB remap + load recording, fp8 activations
 * on MXFP4 experts), as hand-written HIP kernels for gfx950.
 *
 * What the layer is, from the pages:
 *  - The MegaMoEV2 operator runs quant, dispatch, GEMM1, GEMM2 and combine;
 *    its small-input path does all of them in one kernel for up to 512 tokens
 *    per rank, and its persistent large-input path serves extend steps of at
 *    least 1024 tokens [sglang PR 47065 "[Perf] [AMD] dsv4: Use the aiter
 *    MegaMoE small- and large-input paths", intro and Modifications].
 *  - Activations are fp8 and routed experts MXFP4 ("a8w4") [InferenceX PR 3430
 *    "[AMD][MI35X] 0926 DSV4 sglang mtp agentic", Additional detail section].
 *  - Each token picks its top-6 routed experts [sglang PR 35619 "Aiter/FlyDSL
 *    MegaMoEv2 backend for DeepSeek-V4", "Four settings that silently break
 *    it", item 2].
 *  - Prefill fuses the EPLB logical-to-physical remap with load recording
 *    [same page, Summary]; EPLB runs with redundant physical experts
 *    [FlyDSL issue 978 "Investigate MegaMoEV2 end-to-end throughput gap vs V1
 *    on 8xMI355X", Benchmark plan].
 *  The pages print no formula; the readings used for the unstated steps are:
 *  sigmoid scores and renormalised top-k weights, replica = MurmurHash3
 *  fmix32(global token id) mod replica count, e8m0 per-128-column activation
 *  scales, SwiGLU between the GEMMs, routing weights applied in the combine.
 *
 * Conventions for every call
 *  - Pointers other than `dims`, `taps` and `chosen` are DEVICE pointers owned
 *    by the caller; they must be 16-byte aligned.  The library allocates
 *    nothing and keeps no state between calls (moe_forward_noalloc's scratch
 *    is a fixed array of the library's device code, not an allocation).
 *  - Every call is asynchronous on `stream` (NULL = the default stream); it
 *    never synchronises the host and never prints.
 *  - Arguments are validated on the host before any launch; a failed check
 *    returns a negative moe_status_t and launches nothing.  A launch error
 *    becomes MOE_ERR_HIP.  Finite inputs, expert ids in [0, E) and replica
 *    tables whose entries lie in [0, P_total) are the caller's contract.
 *  - T == 0 is valid and launches nothing (the outputs have no rows).
 *  - Calls on one workspace must not overlap in time; use one workspace per
 *    stream for concurrent calls.
 *
 * Layouts (row-major, C order):
 *  logits   f32  [T, E]
 *  x        bf16 [T, H]                 (uint16 bit patterns)
 *  w1       u8   [P_local, 2F, H/2]     MXFP4: e2m1 pairs, element 2i in the low
 *                                       nibble; rows [0, F) gate, [F, 2F) up
 *  w1s      u8   [P_local, 2F, H/32]    e8m0 scale of each 32-element block along K
 *  w2       u8   [P_local, H, F/2]
 *  w2s      u8   [P_local, H, F/32]
 *  pw1, pw1s, pw2, pw2s                 the same weights repacked by
 *                                       moe_pack_weights (sizes: moe_packed_bytes):
 *    each 16-row tile, each 256-wide K step, each of the step's two
 *    16x16x128 MFMAs: 64 lanes x 16 bytes, lane 16g + r holding row r,
 *    32-block 8 step + 4 i + g; scales per tile and 4 steps: 64 lanes x 8
 *    bytes, byte 2 (step % 4) + i of lane 16g + r = scale of row r, block
 *    8 step + 4 i + g.  K is padded with zero blocks to a multiple of 1024.
 *  rep_count  i32 [E]                   replicas of each logical expert (>= 1)
 *  rep_slots  i32 [E, R_max]            physical slot of replica r of expert e
 *  load_hist  i32 [P_total]             += pairs per physical slot (nullable)
 *  topk_ids i32 [T, k], topk_w f32 [T, k], phys_ids i32 [T, k]
 *  counts   i32 [P_local], offsets i32 [P_local + 1]
 *  row_of_pair i32 [T*k] (-1: remote pair), pair_of_row i32 [T_max*k]
 *  xq u8 [T_max*k, H] (fp8 e4m3fn), xs u8 [T_max*k, H/128] (e8m0)
 *  aq u8 [T_max*k, F], as u8 [T_max*k, F/128]
 *  out bf16 [T, H]
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* moe_stream_t; /* a hipStream_t */

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1, /* null pointer, bad shape or misaligned pointer */
  MOE_ERR_UNSUPPORTED = -2, /* a size beyond the limits below */
  MOE_ERR_WORKSPACE = -3,   /* workspace missing or smaller than moe_workspace_bytes */
  MOE_ERR_HIP = -4,         /* a kernel launch failed */
  MOE_ERR_SCRATCH = -5      /* moe_forward_noalloc: the dims need more than its fixed scratch */
} moe_status_t;

typedef enum {
  MOE_PATH_AUTO = 0,    /* SMALL_M if T <= min(small_m_max, 1024), LARGE_M if T >= large_m_min,
                           else STAGED */
  MOE_PATH_SMALL_M = 1, /* four launches in (token, j) pair order: route + remap + quant of every
                           token; GEMM1 and GEMM2 weight streaming, each block listing its slot's
                           pairs itself; combine + load record.  No bucket scan or permute.
                           T <= 1024 (else MOE_ERR_UNSUPPORTED). */
  MOE_PATH_STAGED = 2,  /* the component calls in sequence (bucketed rows, weight streaming) */
  MOE_PATH_LARGE_M = 3  /* bucketed rows, persistent tiled GEMMs once the mean rows per physical
                           slot (T k / P_total) exceed 24, weight streaming below */
} moe_path_t;

/* Problem sizes of one call.  Limits: 0 <= T <= T_max <= 1<<20; H, F
 * multiples of 128, each in [128, 16384]; 1 <= E <= 1024; 1 <= k <= min(E, 16);
 * 1 <= P_total <= 1024; 0 <= p0, 1 <= P_local, p0 + P_local <= P_total;
 * 1 <= R_max <= 64.  Without EPLB: P_total = E, R_max = 1, rep_slots[e] = e. */
typedef struct {
  int32_t T, T_max;
  int32_t H, F, E, k;
  int32_t P_total, p0, P_local, R_max;
  uint32_t token_id_base;  /* global id of token 0; the remap hashes global ids */
  int32_t small_m_max;     /* 0 -> 512  [sglang PR 47065, intro]            */
  int32_t large_m_min;     /* 0 -> 1024 [sglang PR 47065, Modifications]    */
} moe_dims_t;

/* Optional device copies of intermediate results for parity checks, and
 * timing hooks; any member may be NULL.  Shapes as in the layout table above.  Every path
 * writes topk_ids, topk_w, phys_ids, counts and offsets.  STAGED and
 * LARGE_M (bucketed rows) write row_of_pair, pair_of_row, xq, xs, aq, as;
 * SMALL_M writes instead the per-token activations xq_tok u8 [T, H] /
 * xs_tok u8 [T, H/128] (every token, local pairs or not) and the per-pair
 * act rows aq_pair u8 [T*k, F] / as_pair u8 [T*k, F/128] (rows of local
 * pairs only). */
typedef struct {
  int32_t* topk_ids;
  float* topk_w;
  int32_t* phys_ids;
  int32_t* counts;
  int32_t* offsets;
  int32_t* row_of_pair;
  int32_t* pair_of_row;
  uint8_t* xq;
  uint8_t* xs;
  uint8_t* aq;
  uint8_t* as;
  uint8_t* xq_tok;
  uint8_t* xs_tok;
  uint8_t* aq_pair;
  uint8_t* as_pair;
  /* Timing hooks (HOST values: hipEvent_t handles created by the caller, any
   * may be NULL): moe_forward records gemm1_events[0] / [1] on `stream` right
   * before / after its GEMM1 launch and gemm2_events likewise around GEMM2,
   * so that a caller can time those kernels inside the whole forward. */
  void* gemm1_events[2];
  void* gemm2_events[2];
} moe_taps_t;

/* Bytes of device workspace every call below needs for `dims` (sized by
 * T_max, independent of T).  Returns 0 for invalid dims. */
size_t moe_workspace_bytes(const moe_dims_t* dims);

/* The path MOE_PATH_AUTO takes for `dims`: small-input at most small_m_max
 * tokens, large-input from large_m_min tokens, staged in between
 * [sglang PR 47065, intro and Modifications; the aiter commit note on the
 * three-state large-input switch]. */
moe_path_t moe_select_path(const moe_dims_t* dims);

/* Static text for a status code. */
const char* moe_status_string(int status);

/* Bytes of a packed weight buffer for `dims` over all P_local slots:
 * which = 0 pw1, 1 pw1s, 2 pw2, 3 pw2s.  Returns 0 for invalid arguments. */
size_t moe_packed_bytes(const moe_dims_t* dims, int which);

/* Repack MXFP4 expert weights (natural layout above) into the MFMA-operand
 * order the GEMM kernels stream: every weight load of a wavefront becomes one
 * contiguous 1 KB and one 8-byte scale load covers four K steps of a tile.
 * Pure byte movement, run once when weights are loaded (like the checkpoint
 * conversion that produced the MXFP4 experts [InferenceX PR 3430, Additional
 * detail section]).  Output buffers must not overlap the inputs. */
int moe_pack_weights(const moe_dims_t* dims, const uint8_t* w1, const uint8_t* w1s, const uint8_t* w2,
                     const uint8_t* w2s, uint8_t* pw1, uint8_t* pw1s, uint8_t* pw2, uint8_t* pw2s,
                     moe_stream_t stream);

/* a1. Top-k routing [sglang PR 35619, "Four settings that silently break it"].
 * For each token: the k largest logits (descending, equal logits to the lower
 * expert id); weight_j = sigmoid(l_j) / sum_i sigmoid(l_i) in f32. */
int moe_route(const moe_dims_t* dims, const float* logits, int32_t* topk_ids, float* topk_w,
              moe_stream_t stream);

/* a2. EPLB logical -> physical remap with load recording [sglang PR 35619,
 * Summary; FlyDSL issue 978, Data-quality gates].
 * phys[t][j] = rep_slots[e][fmix32(token_id_base + t) mod rep_count[e]],
 * e = topk_ids[t][j]; if load_hist != NULL, load_hist[p] += number of pairs
 * with phys == p (all T*k pairs, every slot).  Deterministic, no atomics. */
int moe_eplb_remap_record(const moe_dims_t* dims, const int32_t* topk_ids, const int32_t* rep_count,
                          const int32_t* rep_slots, int32_t* phys_ids, int32_t* load_hist,
                          void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* The replica a2 sends a token to (host utility, no device call): the index
 * r in [0, rep_count) of rep_slots[e][r] for global token id `token_id` of an
 * expert with `rep_count` replicas, r = fmix32(token_id) mod rep_count
 * (MurmurHash3's 32-bit finaliser).  The kernels use the same rule; a
 * rep_count outside [1, R_max] (a broken table) is clamped into that range
 * there and here, so that no table read leaves the expert's row. */
int32_t moe_replica_of(uint32_t token_id, int32_t rep_count, int32_t R_max);

/* a3 + a4. Bucket this GPU's pairs by local slot and quantise + dispatch the
 * activations [sglang PR 47065, intro: "quant, dispatch"].
 * Local pairs have p0 <= phys < p0 + P_local; slot s = phys - p0 owns rows
 * [offsets[s], offsets[s+1]), filled in ascending (t, j).  Row r holds token
 * pair_of_row[r] / k quantised per 128 columns: scale byte e + 127 with e the
 * smallest integer such that amax <= 448 * 2^e, codes RNE_e4m3fn(x * 2^-e). */
int moe_quant_permute(const moe_dims_t* dims, const uint16_t* x, const int32_t* phys_ids,
                      uint8_t* xq, uint8_t* xs, int32_t* counts, int32_t* offsets,
                      int32_t* row_of_pair, int32_t* pair_of_row,
                      void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* a5. GEMM1 + SwiGLU + fp8 requant, grouped by slot [sglang PR 47065, intro].
 * For each row r of slot s: h = W1_s a_r (f32 accumulation of block-scaled
 * fp8 x MXFP4 products); act_f = silu(h_f) * h_{F+f}; act requantised with
 * the a4 rule per 128 columns into aq / as.  `offsets` as from a3; weights
 * packed by moe_pack_weights. */
int moe_grouped_gemm1_swiglu(const moe_dims_t* dims, const uint8_t* xq, const uint8_t* xs,
                             const int32_t* offsets, const uint8_t* pw1, const uint8_t* pw1s,
                             uint8_t* aq, uint8_t* as, void* workspace, size_t workspace_bytes,
                             moe_stream_t stream);

/* a6 + a7. GEMM2 and the routing-weighted combine [sglang PR 47065, intro].
 * y_r = W2_s dequant(aq_r) (f32); out[t] = bf16_rne(sum over local j, ascending,
 * of topk_w[t][j] * y[row_of_pair[t*k+j]]); tokens with no local pair get +0. */
int moe_grouped_gemm2_combine(const moe_dims_t* dims, const uint8_t* aq, const uint8_t* as,
                              const int32_t* offsets, const uint8_t* pw2, const uint8_t* pw2s,
                              const int32_t* row_of_pair, const float* topk_w, uint16_t* out,
                              void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* a5 on the small-input path's pair-indexed rows (what MOE_PATH_SMALL_M runs
 * between its front end and GEMM2) [sglang PR 47065, intro].  Same arithmetic
 * as moe_grouped_gemm1_swiglu; the rows of slot s are the pairs p (ascending)
 * with phys_ids[p] == p0 + s, listed by each block itself.  Inputs: per-token
 * activations xq_tok u8 [T, H] / xs_tok u8 [T, H/128] (the a4 rule) and
 * phys_ids [T*k]; outputs: act rows aq_pair u8 [T*k, F] / as_pair
 * u8 [T*k, F/128] (rows of local pairs only; others untouched) and
 * counts i32 [P_local].  T <= 1024, else MOE_ERR_UNSUPPORTED.  No workspace. */
int moe_grouped_gemm1_swiglu_pairs(const moe_dims_t* dims, const uint8_t* xq_tok, const uint8_t* xs_tok,
                                   const int32_t* phys_ids, const uint8_t* pw1, const uint8_t* pw1s,
                                   uint8_t* aq_pair, uint8_t* as_pair, int32_t* counts, moe_stream_t stream);

/* a6 + a7 on pair-indexed rows: y_p = W2_s dequant(aq_pair_p) for every local
 * pair p (f32, in the workspace), then out as in moe_grouped_gemm2_combine
 * with row(t, j) = t*k + j; `offsets` i32 [P_local + 1] receives the
 * exclusive scan of `counts`.  T <= 1024, else MOE_ERR_UNSUPPORTED. */
int moe_grouped_gemm2_combine_pairs(const moe_dims_t* dims, const uint8_t* aq_pair, const uint8_t* as_pair,
                                    const int32_t* phys_ids, const uint8_t* pw2, const uint8_t* pw2s,
                                    const float* topk_w, const int32_t* counts, int32_t* offsets, uint16_t* out,
                                    void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* The whole layer, a1..a7, on `path` (MOE_PATH_AUTO: moe_select_path).
 * rep_count / rep_slots describe the replica table; load_hist (nullable) is
 * accumulated as in a2 (pass NULL in decode: recording is prefill-only
 * [sglang PR 35619, Summary]).  `chosen` (host, nullable) receives the path
 * taken.  `taps` (host struct of device pointers, nullable) receives copies
 * of the intermediates. */
int moe_forward(const moe_dims_t* dims, moe_path_t path, const uint16_t* x, const float* logits,
                const uint8_t* pw1, const uint8_t* pw1s, const uint8_t* pw2, const uint8_t* pw2s,
                const int32_t* rep_count, const int32_t* rep_slots, int32_t* load_hist,
                uint16_t* out, const moe_taps_t* taps, moe_path_t* chosen,
                void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* a16w4 variant of the whole layer: bf16 activations on the MXFP4 experts,
 * no activation quantisation (the pages' non-EP arms run the MXFP4 experts
 * with bf16 activations [InferenceX PR 3430, Additional detail section]).
 * Routing, remap + record and buckets as moe_forward; GEMM1 takes each
 * bucketed row's bf16 input row as is (products exact, f32 accumulation),
 * act = silu(gate) * up rounded to bf16 (nearest even), GEMM2 on the bf16
 * act, combine as moe_forward.  The weight scale bytes of non-zero MXFP4
 * elements must lie in [2, 252] (every value then a normal bf16; the caller's
 * contract like finite inputs).  Rows: T <= 1024 takes pair-indexed rows as
 * MOE_PATH_SMALL_M (four launches), larger T bucketed rows as the staged
 * path (seven launches).  taps (nullable): topk_ids, topk_w, phys_ids,
 * counts, offsets as moe_forward, and for bucketed rows also row_of_pair,
 * pair_of_row (other members ignored); act_tap (nullable, device): bf16 act
 * rows [T_max*k, F], in bucket order for bucketed rows, by pair t*k+j for
 * pair-indexed rows (rows of remote pairs unspecified).  Workspace:
 * moe_a16w4_workspace_bytes(dims).  T * H * 2 and T_max * k * F * 2 bytes
 * must stay below 2^31 (else MOE_ERR_UNSUPPORTED).  Asynchronous on
 * `stream`. */
size_t moe_a16w4_workspace_bytes(const moe_dims_t* dims);
int moe_forward_a16w4(const moe_dims_t* dims, const uint16_t* x, const float* logits, const uint8_t* pw1,
                      const uint8_t* pw1s, const uint8_t* pw2, const uint8_t* pw2s, const int32_t* rep_count,
                      const int32_t* rep_slots, int32_t* load_hist, uint16_t* out, const moe_taps_t* taps,
                      uint16_t* act_tap, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* The small-input path with the token count on the device, for captured
 * graphs: decode graphs are captured per token-count bucket and must also
 * run idle (zero-token) steps [sglang PR 35619, Summary: graph-safe idle
 * handling; sglang PR 47065, Modifications: DP-synchronised buckets for the
 * captured graphs, forward_small_m(max_tokens=)].  dims->T is the bucket
 * capacity (<= 1024; every launch shape follows it); num_tokens (DEVICE, i32,
 * 4-byte aligned) holds the step's valid count n, read by the kernels, so one
 * capture serves every n in [0, dims->T] (values outside are clamped).  The
 * first n tokens go through the layer exactly as moe_forward(MOE_PATH_SMALL_M)
 * with T = n computes them; rows [n, T) of `out` are written as +0; load_hist
 * (nullable) counts only the first n tokens' pairs; taps hold the first n
 * tokens' intermediates (phys_ids of the others = -1, the rest unspecified).
 * Other arguments and errors as moe_forward.  Launches no memset and
 * allocates nothing, so the four launches can be captured into a graph. */
int moe_forward_small_m(const moe_dims_t* dims, const int32_t* num_tokens, const uint16_t* x, const float* logits,
                        const uint8_t* pw1, const uint8_t* pw1s, const uint8_t* pw2, const uint8_t* pw2s,
                        const int32_t* rep_count, const int32_t* rep_slots, int32_t* load_hist, uint16_t* out,
                        const moe_taps_t* taps, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* Router projection in front of a1: logits[t][e] = sum_k x[t][k] w_gate[e][k]
 * (bf16 x bf16 products, f32 accumulation in an unspecified order).  The
 * gate is stored in BF16 [InferenceX PR 3430, Additional detail section];
 * routing then takes the top-k of these logits (moe_route / moe_forward).
 * Layouts: x bf16 [T, H] (as everywhere), w_gate bf16 [E, H] (one row per
 * logical expert, no bias), logits f32 [T, E].  Only dims->T, T_max, H, E
 * matter (the other fields must still be valid dims).  Workspace: at least
 * moe_router_workspace_bytes(dims) bytes, 256-byte aligned (split-K partial
 * sums; sized by T_max).  T == 0 launches nothing.  Asynchronous on `stream`;
 * one or two launches. */
size_t moe_router_workspace_bytes(const moe_dims_t* dims);
int moe_router_logits(const moe_dims_t* dims, const uint16_t* x, const uint16_t* w_gate, float* logits,
                      void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* EPLB rebalance: a new replica table from the loads recorded by a2 (host
 * call; every pointer is a HOST pointer; no stream, no device memory).
 * The pages run EPLB with redundant physical experts and rebalance every few
 * hundred steps from the recorded per-expert loads [sglang PR 35619,
 * Summary and reviewer reproduction; FlyDSL issue 978, Benchmark plan and
 * Data-quality gates]; they give no placement algorithm.  This one:
 *  1. L_e = sum of load_hist[s] over the slots s with slot_expert_old[s] == e
 *     (slots holding -1 are ignored);
 *  2. every expert gets one replica; P_total - E times, the expert with the
 *     largest L_e / c_e (exact comparison) among those with c_e < R_max gets
 *     one more, equal shares to the lower e;
 *  3. replicas in descending L_e / c_e (then e, then replica index) go one by
 *     one to the rank (slots [r P_total/n_ranks, (r+1) P_total/n_ranks)) with
 *     a free slot that does not hold e yet, else any rank with a free slot,
 *     the one with the smallest load (f64 sum of the shares placed on it,
 *     in placement order), then the lower rank;
 *  4. inside a rank a replica keeps a slot that held e in the old map (the
 *     lowest first), so that it needs no migration; the others fill the
 *     rank's remaining slots in ascending order, in placement order.
 * Inputs: load_hist i32 [P_total] (>= 0; the histogram of all ranks' tokens
 * in a multi-GPU job), slot_expert_old i32 [P_total] (expert of each slot,
 * -1 = empty).  Outputs: rep_count i32 [E], rep_slots i32 [E, R_max] (each
 * expert's slots ascending, -1 padded; the table moe_forward takes with this
 * R_max), slot_expert_new i32 [P_total].  Requires E <= P_total,
 * P_total % n_ranks == 0 and E * R_max >= P_total; MOE_ERR_INVALID_ARG
 * otherwise (nothing written). */
int moe_eplb_rebalance(int32_t E, int32_t P_total, int32_t n_ranks, int32_t R_max, const int32_t* load_hist,
                       const int32_t* slot_expert_old, int32_t* rep_count, int32_t* rep_slots,
                       int32_t* slot_expert_new);

/* EPLB weight migration for this GPU's slots (the pages' data-quality gates
 * check that rebalances and migrations take place [FlyDSL issue 978,
 * Data-quality gates]).  For each local slot s
 * (s < dims->P_local) with src_expert[s] >= 0, the packed weights of slot s
 * (pw1, pw1s, pw2, pw2s, layout of moe_pack_weights) become a byte copy of
 * logical expert src_expert[s]'s packed weights in the pool; slots with -1
 * keep their bytes.  The pool holds n_pool experts packed by moe_pack_weights
 * (a pack with P_local = n_pool): on one GPU it stands in for the peer or
 * host memory a multi-GPU job would fetch experts from.  src_expert: DEVICE
 * i32 [P_local]; entries >= n_pool are skipped.  Only dims->H, F, P_local
 * matter; the pool and the slots must not overlap.  Asynchronous on
 * `stream`, one launch. */
int moe_eplb_migrate(const moe_dims_t* dims, const int32_t* src_expert, int32_t n_pool, const uint8_t* pool_pw1,
                     const uint8_t* pool_pw1s, const uint8_t* pool_pw2, const uint8_t* pool_pw2s, uint8_t* pw1,
                     uint8_t* pw1s, uint8_t* pw2, uint8_t* pw2s, moe_stream_t stream);

/* moe_forward without a workspace argument, for callers that cannot allocate
 * device memory (code under graph capture, tight serving loops, harnesses
 * that forbid hipMalloc).  Same arguments, paths, results and errors as
 * moe_forward with taps = NULL; the workspace is instead a fixed device
 * array of MOE_NOALLOC_SCRATCH_BYTES inside the library, one per GPU, that
 * each GPU the library runs on holds until the process ends.  The first call
 * on a device resolves that device's copy (the calling thread's current
 * device must be the stream's device).  Dims whose moe_workspace_bytes exceed
 * the scratch return MOE_ERR_SCRATCH before any launch (at d_model 7168,
 * d_ff 2048, top-6: T_max up to 587 tokens).  The call allocates nothing and
 * needs no part of the scratch to start at zero (every kernel writes what it
 * reads), but all calls on one GPU share that GPU's scratch, which keeps the
 * last call's contents: calls that overlap in time on one GPU (other streams,
 * other threads) race and must be serialised by the caller. */
#define MOE_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)
int moe_forward_noalloc(const moe_dims_t* dims, moe_path_t path, const uint16_t* x, const float* logits,
                        const uint8_t* pw1, const uint8_t* pw1s, const uint8_t* pw2, const uint8_t* pw2s,
                        const int32_t* rep_count, const int32_t* rep_slots, int32_t* load_hist, uint16_t* out,
                        moe_path_t* chosen, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * Linear operators: the fp8 product with an f32 scale per block of 128 (the
 * format of fp8 checkpoints' dense, shared-expert and routed-expert layers),
 * the quantiser in front of it, and the 16-bit products grouped by expert
 * with both gradients (fine-tuning of unquantised experts).
 *
 * Groups.  Weights hold `groups` matrices [N, K]; rows [offsets[g],
 * offsets[g+1]) of the row tensors belong to matrix g.  offsets: DEVICE i32
 * [groups + 1], ascending, within [0, rows] (the caller's contract; entries
 * outside are clamped, so nothing outside the tensors is touched).  NULL is
 * allowed for groups == 1 and means all rows.  Groups may be empty.  Rows in
 * no group are not written by the row products.  moe_quant_permute's
 * `offsets` are such offsets.  `rows` may be a capacity, as there, but how the
 * work is divided is chosen for `rows` rows: the closer, the faster.
 * Sums and scales are f32; each output is rounded once, to nearest even.
 * Results do not depend on timing: there are no atomic sums.
 * Conventions as above (device pointers, 16-byte alignment, asynchronous on
 * `stream`, nothing allocated, host validation first).  rows == 0 is valid;
 * row tensors may then be NULL.  Outputs must not overlap inputs.
 * ------------------------------------------------------------------------- */
typedef enum {
  MOE_TYPE_BF16 = 0,
  MOE_TYPE_F16 = 1,
  MOE_TYPE_F32 = 2,
  MOE_TYPE_FP8 = 3 /* e4m3fn codes */
} moe_type_t;

/* Limits: 0 <= rows <= 1<<20, 1 <= N, K <= 32768, 1 <= groups <= 1024.
 * in_type FP8: K a multiple of 16, any N, out_type BF16, F16 or F32.
 * in_type BF16 or F16: K a multiple of 8 (and N for the gradients), out_type
 * in_type or F32. */
typedef struct {
  int32_t rows, N, K, groups;
  int32_t in_type, out_type; /* moe_type_t */
} moe_linear_t;

/* Workspace bytes of any linear call on these sizes, the gradients included
 * (independent of out_type).  May be 0; returns 0 for invalid sizes too.  It is
 * no bound for fewer rows, which may need more: split reductions are for few. */
size_t moe_linear_workspace_bytes(const moe_linear_t* d);

/* q u8 [rows, K] = e4m3_rne(x * (1 / s)), qs f32 [rows, ceil(K/128)]:
 * s = max(amax / 448, 2^-126) over the row's block of 128 columns (the last
 * one may be shorter), all in f32.  x: BF16, F16 or F32 (x_type) [rows, K], ldx
 * elements between rows; K and ldx multiples of 16 (K at most 32768).  A block
 * holding a NaN gets a NaN scale and NaN codes; one holding an infinity an
 * infinite scale, zero codes and NaN at the infinity. */
int moe_fp8_quant(int32_t rows, int32_t K, int32_t x_type, const void* x, int64_t ldx, uint8_t* q, float* qs,
                  moe_stream_t stream);

/* The same of h = silu(x[:, :K]) * x[:, K:2K] in f32; x [rows, 2K], ldx >= 2K.
 * h keeps its value where silu alone leaves f32's normal range (gates below
 * -87) and a large x[:, K:2K] brings the product back. */
int moe_fp8_swiglu_quant(int32_t rows, int32_t K, int32_t x_type, const void* x, int64_t ldx, uint8_t* q, float* qs,
                         moe_stream_t stream);

/* y[r, n] = sum over blocks b of 128 columns of
 *   xs[r, b] * ws[g, n/128, b] * sum_{k in b} xq[r, k] w[g, n, k].
 * xq u8 [rows, K], xs f32 [rows, ceil(K/128)], w u8 [groups, N, K], ws f32
 * [groups, ceil(N/128), ceil(K/128)], y [rows, N] of out_type.  d->in_type FP8.
 * Inside a block the matrix instruction aligns 32 products to the largest of
 * them and keeps about 14 bits below its leading one; everything after is f32,
 * the product xs * ws first (below 2^-126 it loses bits). */
int moe_fp8_linear(const moe_linear_t* d, const uint8_t* xq, const float* xs, const uint8_t* w, const float* ws,
                   const int32_t* offsets, void* y, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* y[r, n] = sum_k x[r, k] w[g, n, k]: x [rows, K] and w [groups, N, K] of
 * in_type, y [rows, N] of out_type. */
int moe_grouped_linear(const moe_linear_t* d, const void* x, const void* w, const int32_t* offsets, void* y,
                       void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* Gradient of the rows: dx[r, k] = sum_n dy[r, n] w[g, n, k]; dy [rows, N] of
 * in_type, dx [rows, K] of out_type. */
int moe_grouped_linear_dx(const moe_linear_t* d, const void* dy, const void* w, const int32_t* offsets, void* dx,
                          void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* Gradient of the weights: dw[g, n, k] = sum over the group's rows of
 * dy[r, n] x[r, k] (zeros for an empty group); dw [groups, N, K] of out_type,
 * overwritten. */
int moe_grouped_linear_dw(const moe_linear_t* d, const void* dy, const void* x, const int32_t* offsets, void* dw,
                          void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * What a product by expert is followed by, and the gradient through it.  16-bit
 * operands (in_type BF16 or F16); sizes, groups and conventions as above.
 *   z = x w_g^T + b_g,   y = act(z) + residual                     (gated 0)
 *                        y = act(z[:, :F]) * z[:, F:] + residual   (gated 1, N = 2 F)
 * ------------------------------------------------------------------------- */
typedef enum {
  MOE_ACT_NONE = 0,
  MOE_ACT_RELU = 1,
  MOE_ACT_SILU = 2,     /* z / (1 + e^-z); gated: SwiGLU */
  MOE_ACT_GELU = 3,     /* z Phi(z) */
  MOE_ACT_GELU_TANH = 4 /* 0.5 z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) */
} moe_act_t;

/* Workspace bytes of the two calls below on these sizes (any activation).  May
 * be 0; 0 for invalid sizes too.  No bound for fewer rows, which may need more. */
size_t moe_linear_act_workspace_bytes(const moe_linear_t* d);

/* The product with its epilogue.  x [rows, K], w [groups, N, K] and bias [groups,
 * N] (nullable) of in_type; residual (nullable) and y [rows, N], gated [rows,
 * N / 2], of out_type; pre (nullable) [rows, N] of out_type receives z, for the
 * gradient.  N must be even if gated.  residual may be y itself.  The sum, bias,
 * activation and residual are f32, y and z each rounded once (y is not made from
 * the rounded z).  Rows in no group are not written, in y and in pre.  An
 * infinite z gives what the formula gives: NaN where it has 0 * infinity. */
int moe_grouped_linear_act(const moe_linear_t* d, int32_t act, int32_t gated, const void* x, const void* w,
                           const void* bias, const void* residual, const int32_t* offsets, void* y, void* pre,
                           void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* The gradient through bias and activation, for dy = dL/dy and z = pre:
 *   dz = dy act'(z),  gated: (dy z[:, F:] act'(z[:, :F]), dy act(z[:, :F]));
 *   db_g = sum over the group's rows of dz (zeros for an empty group).
 * dy [rows, N], gated [rows, N / 2], and pre [rows, N] of out_type; dz [rows, N]
 * of in_type, what moe_grouped_linear_dx and _dw take as dy; db (nullable) f32
 * [groups, N], overwritten, added up from the f32 values before their rounding.
 * (The residual's gradient is dy.)  relu'(0) = 0.  An infinite z gives what the
 * formulas give, as above: NaN for silu, gelu and gelu_tanh, but act(inf) = inf.  N
 * a multiple of 8; K is not used but must be valid.  dz may be pre itself where the
 * types are the same.  The workspace is needed for db alone.  One launch; for db of more rows than
 * a few blocks can add up (256 at most), two. */
int moe_grouped_linear_act_backward(const moe_linear_t* d, int32_t act, int32_t gated, const void* dy, const void* pre,
                                    const int32_t* offsets, void* dz, float* db, void* workspace,
                                    size_t workspace_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * The global gradient norm and clipping by it.  `tensors` is a HOST array that
 * is read during the call alone; its pointers are device pointers, aligned to
 * their element.  Captured into a graph, a call keeps the addresses that it was
 * given.  The workspace (moe_grad_workspace_bytes(count), 16-byte aligned) is
 * needed by every call.  Sums are f64 and added in a fixed order.
 * ------------------------------------------------------------------------- */
#define MOE_GRAD_MAX_TENSORS 65536
typedef struct {
  const void* in;
  void* out;    /* moe_grad_clip writes here; may be its own `in`, else no outputs and inputs overlap.
                   moe_grad_norm: not used */
  int64_t n;    /* elements, 0 to 2^36 */
  int32_t type; /* BF16, F16 or F32, of both */
  int32_t reserved;
} moe_tensor_t;

size_t moe_grad_workspace_bytes(int32_t count);

/* norm f32 [1] (device, 4-byte aligned) = sqrt(sum over all tensors of in^2).
 * ceil(count / 168) + 1 launches. */
int moe_grad_norm(const moe_tensor_t* tensors, int32_t count, float* norm, void* workspace, size_t workspace_bytes,
                  moe_stream_t stream);

/* out = in * min(1, max_norm / (norm + 1e-6)), the factor and the product in f64,
 * rounded to f32 and from there to a 16-bit type; norm (nullable, f32) receives the
 * norm before.  max_norm >= 0.  A NaN among the values makes every output NaN; an
 * infinity makes the factor 0 (and itself NaN).  2 ceil(count / 168) launches. */
int moe_grad_clip(const moe_tensor_t* tensors, int32_t count, float max_norm, float* norm, void* workspace,
                  size_t workspace_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * The whole layer, a1..a7, on unquantised experts for a few tokens: a16w16.
 * Routing, remap and record as moe_forward; then for each local pair (t, j),
 * e its slot,  h = w1_e x_t,  act = silu(h[:F]) * h[F:],  out_t = sum over j of
 * topk_w[t][j] w2_e act.  x and out [T, H], w1 [P_local, 2F, H] and w2 [P_local,
 * H, F] of `type` (BF16 or F16), in their natural layout, as moe_grouped_linear
 * takes them.  Sums, activation, weights and topk_w * act are f32 (F16: of 64
 * columns in a row, the second product takes what is above 2^-38 of the largest),
 * and out is rounded once.
 * Tokens with no local pair get +0.  T <= 32, else MOE_ERR_UNSUPPORTED (more
 * tokens: moe_quant_permute's buckets with moe_grouped_linear_act).
 * num_tokens (nullable, DEVICE i32, 4-byte aligned): the step's token count n,
 * read by the kernels and clamped to [0, T], for captured graphs as in
 * moe_forward_small_m: rows [n, T) of out are +0, load_hist counts the first n.
 * taps (nullable): topk_ids, topk_w and phys_ids are written for the first n
 * tokens (phys_ids of the others: -1), other members ignored.  Workspace:
 * moe_a16w16_workspace_bytes(dims), 256-byte aligned.  Two launches.
 * ------------------------------------------------------------------------- */
size_t moe_a16w16_workspace_bytes(const moe_dims_t* dims);
int moe_forward_a16w16(const moe_dims_t* dims, int32_t type, const int32_t* num_tokens, const void* x,
                       const float* logits, const void* w1, const void* w2, const int32_t* rep_count,
                       const int32_t* rep_slots, int32_t* load_hist, void* out, const moe_taps_t* taps, void* workspace,
                       size_t workspace_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
