/*
 * mi355moe.h -- C ABI of the MXFP8 x MXFP4 fused MoE expert layer for AMD
 * Instinct MI355X (gfx950).
 *
 * The layer (one GPU's share of a Kimi-K3-style routed-expert MoE) is five
 * calls, issued in this order on one HIP stream (the first three can also be
 * issued as one, moe_route_quant_permute; with top-k ids computed elsewhere,
 * the second and third as one, moe_quant_permute):
 *
 *   moe_route        sigmoid + correction-bias top-k routing, renormalised weights
 *   moe_quant_mxfp8  bf16 activations -> MXFP8 (E4M3 + one E8M0 scale per 32)
 *   moe_permute      group the kept routes by local expert (stable)
 *   moe_fc1_situ     grouped FC1 (MXFP8 x MXFP4) + SiTU + requantisation to MXFP8
 *   moe_fc2_combine  grouped FC2 (MXFP8 x MXFP4) + top-k weighted combine to bf16
 *
 * Sources (the pages this library implements): page 1 = the SM120 FlashInfer
 * MXFP4 experiment log for Kimi-K3 (sections "Serving call chain", "Key
 * sources" table, "Real checkpoint contract", "TP/EP expert mapping", "Phase 2
 * correctness harness", "NaN/Inf decision record"); page 5 = the Kimi-K3 MoE
 * path notes (weight/scale layouts, symmetric buffer views, pre-dispatch
 * quantisation).
 *
 * Conventions for every call:
 *  - Every pointer is a DEVICE pointer owned by the caller.  The library never
 *    allocates, frees or synchronises; every call is asynchronous on `stream`
 *    (0 = the null stream) and keeps no state between calls.
 *  - Arguments are validated before anything is launched.  A failed check
 *    returns a status and launches nothing; the pure argument checks make no
 *    HIP call, so they can be exercised on a machine without a GPU.  The
 *    device check (gfx950) runs after them.  A launch failure returns
 *    MOE_ERR_HIP.  Nothing retries or falls back to another path.
 *  - Pointers to byte / bf16 tensors must be 16-byte aligned; float and int32
 *    tensors 4-byte aligned.
 *  - Shapes: H and I multiples of 128; 1 <= top_k <= min(E, 64); E <= 4096;
 *    1 <= E_local <= 4096; T >= 0 (with T = 0 nothing is launched, except
 *    that moe_permute still writes zero expert offsets).
 *  - Byte layouts (little-endian, row-major):
 *      E4M3  OCP 8-bit float "fn": bias 7, max 448, no infinities.
 *      E2M1  4-bit float: magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6; two per byte,
 *            element 2j in the low nibble of byte j (page 1: packed FP4,
 *            two elements per byte; shapes [rows, K/2]).
 *      E8M0  byte b is 2^(b-127); 0xFF is NaN (page 1, NaN/Inf record).
 *    One scale per 32 consecutive elements along the contraction axis,
 *    stored [rows, K/32] (page 1 checkpoint shapes; page 5 w13 scale
 *    [E, 2I, H/32]).  The activation scale bytes [T, H/32] are the same bytes
 *    as page 5's x_sf view [T, H/128] of int32 words.
 */
#ifndef MI355MOE_H
#define MI355MOE_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 3

/* Status codes have fixed values (page 1 records a Python/C++ enum mismatch
 * that silently turned SiTU into a non-gated activation; these values never
 * change within an ABI version). */
typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_NULL = 1,            /* a required pointer is NULL */
  MOE_ERR_SHAPE = 2,           /* a size or stride is out of range */
  MOE_ERR_ALIGN = 3,           /* a pointer or stride is misaligned */
  MOE_ERR_ENUM = 4,            /* an enum argument has no defined value */
  MOE_ERR_WORKSPACE = 5,       /* workspace too small */
  MOE_ERR_HIP = 6,             /* a HIP runtime call or launch failed */
  MOE_ERR_UNSUPPORTED_DEVICE = 7, /* current device is not gfx950 */
  MOE_ERR_SCRATCH_LIMIT = 8    /* sizes need more than the library's static scratch
                                  (moe_permute_noalloc only) */
} moe_status_t;

/* How moe_fc2_combine sums the top-k FC2 rows of a token (fixed values).
 * Page 1 ("Serving call chain": finalize after GEMM2; "Phase 2 correctness
 * harness" / symmetry constraints) describes both: a fused finalize that
 * accumulates with atomics, whose order and so whose float rounding vary
 * from run to run, and the non-fused finalize kept for bitwise-repeatable
 * results.
 *   MOE_COMBINE_DETERMINISTIC  FC2 writes each kept route's row to the
 *       workspace; a second kernel sums a token's rows in slot order.
 *       Bitwise repeatable.  The default.
 *   MOE_COMBINE_ATOMIC  the FC2 epilogue adds topk_w * row into a float
 *       [T, H] sum in the workspace with atomic adds (cleared first in the
 *       same call), then one pass rounds it to bf16.  Same bar against the
 *       definition, not bitwise repeatable. */
typedef enum moe_combine {
  MOE_COMBINE_DETERMINISTIC = 0,
  MOE_COMBINE_ATOMIC = 1
} moe_combine_t;

/* MOE_ABI_VERSION of the loaded library. */
int moe_abi_version(void);

/* Static description of a status code (never NULL). */
const char* moe_strerror(int status);

/* Bytes of workspace that moe_permute, moe_fc1_situ and moe_fc2_combine need
 * for a layer call with these sizes and combine mode (one buffer serves all
 * three; moe_permute writes the FC kernels' tile schedule into it and
 * moe_fc2_combine keeps the per-route FC2 rows, or with MOE_COMBINE_ATOMIC the
 * float [T, H] sums, there, so pass the same buffer to all three).
 * Returns 0 for invalid sizes or an unknown mode. */
size_t moe_workspace_size(int T, int top_k, int E_local, int H, int I, int mode);

/* a1 -- routing (page 1 "Serving call chain": sigmoid + correction bias +
 * top-k + renormalise; "Key sources" routing row: the bias only selects, the
 * weights come from the bias-free sigmoid scores, normalised; page 5: routed
 * scaling factor).
 *   logits  float [T, E], row stride ld_logits (>= E) elements.
 *   bias    float [E] correction bias, or NULL for none.
 *   s_e = float(sigmoid(logit) evaluated in double); key_e = s_e + bias_e in
 *   float; the top_k largest keys, equal keys ranked by lower expert index,
 *   slots ordered by key descending; w_k = s_k / sum_j s_j (double) times
 *   routed_scaling, rounded to float.
 *   topk_idx int32 [T, top_k] global expert ids; topk_w float [T, top_k].
 *   A NaN logit (or bias) gives a NaN key, which ranks below every other key
 *   (NaN experts are chosen last, lower index first); if one is chosen, the
 *   token's weights are NaN. */
moe_status_t moe_route(const float* logits, int64_t ld_logits, const float* bias,
                       int T, int E, int top_k, float routed_scaling,
                       int32_t* topk_idx, float* topk_w, hipStream_t stream);

/* a2 -- MXFP8 quantisation of bf16 activations (page 5 pre-dispatch step:
 * absmax per 32 elements -> UE8M0 scale -> E4M3; page 1 NaN/Inf record:
 * saturating finite conversion).
 *   x   bf16 bits [T, H], row stride ld_x (>= H, multiple of 8) elements.
 *   Per 32-element group: scale exponent e = the smallest integer with
 *   absmax <= 448 * 2^e, clamped to [-127, 127] (0 for an all-zero group
 *   gives e = -127); element = nearest E4M3 to x * 2^-e, ties to even,
 *   saturating at +-448, sign of zero kept; NaN elements are ignored by the
 *   absmax and encode as 0x00; a group holding +-Inf gets e = 127.
 *   xq  uint8 E4M3 [T, H]; xs  uint8 E8M0 [T, H/32].  H % 32 == 0 suffices
 *   for this call. */
moe_status_t moe_quant_mxfp8(const uint16_t* x, int64_t ld_x, int T, int H,
                             uint8_t* xq, uint8_t* xs, hipStream_t stream);

/* a3 -- grouping by local expert (page 1 "TP/EP expert mapping": a GPU holds
 * the contiguous experts [expert_offset, expert_offset + E_local) and maps
 * global ids into that window; "Phase 2" coverage: -1 masked slots, empty
 * experts).
 *   topk_idx       int32 [T, top_k] global ids (-1 = masked slot).
 *   Route r = t * top_k + k is kept iff its id lies in the window.
 *   expert_offsets int32 [E_local + 1]: rows of local expert e are
 *                  [expert_offsets[e], expert_offsets[e+1]).
 *   sorted_route   int32 [T * top_k]: kept routes in grouped order, ascending
 *                  r within an expert; entries past the kept count are -1.
 *   route_row      int32 [T * top_k]: grouped row of route r, or -1 if dropped.
 *   workspace      >= moe_workspace_size(...) bytes, 256-byte aligned; also
 *                  receives the tile schedule read by the FC calls. */
moe_status_t moe_permute(const int32_t* topk_idx, int T, int top_k, int expert_offset,
                         int E_local, int32_t* expert_offsets, int32_t* sorted_route,
                         int32_t* route_row, void* workspace, size_t ws_bytes,
                         hipStream_t stream);

/* moe_permute without a workspace, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc).  Same arguments as moe_permute minus the workspace, and
 * the same expert_offsets / sorted_route / route_row bytes.  It allocates
 * nothing: the grouping's tile schedule and chunked histogram go to a
 * library-owned device array of 4 MiB (4194304 bytes) that every GPU the
 * library runs on holds until the process ends.
 * Sizes whose schedule does not fit (the schedule part of
 * moe_workspace_size: about 4 * (3 * E_local + T * top_k / 32) bytes plus
 * 4 * E_local bytes per 256 or 512 routes above 2048 routes) return
 * MOE_ERR_SCRATCH_LIMIT before anything is launched.  Every call on one GPU
 * shares that GPU's array, so calls that overlap on one GPU (several streams
 * or threads) race; the FC calls cannot use this call's schedule (they read
 * the one moe_permute writes into their workspace). */
moe_status_t moe_permute_noalloc(const int32_t* topk_idx, int T, int top_k, int expert_offset,
                                 int E_local, int32_t* expert_offsets, int32_t* sorted_route,
                                 int32_t* route_row, hipStream_t stream);

/* a1 + a2 + a3 in one call (decode latency: page 1 "Serving call chain" runs
 * routing, quantisation and grouping before the expert GEMMs; their fixed
 * launch costs are a visible share of a decode step).  Computes exactly what
 * moe_route, then moe_quant_mxfp8, then moe_permute compute with the same
 * arguments (same bytes in every output and in the workspace), and accepts
 * what those three accept together (every check of each; xs needs only
 * 4-byte alignment as in moe_quant_mxfp8).  For T <= 16, E <= 1024 and small
 * enough E_local it is a single launch; otherwise it issues the three
 * launches in order on `stream`. */
moe_status_t moe_route_quant_permute(const float* logits, int64_t ld_logits, const float* bias,
                                     int T, int E, int top_k, float routed_scaling,
                                     const uint16_t* x, int64_t ld_x, int H, int expert_offset,
                                     int E_local, int32_t* topk_idx, float* topk_w, uint8_t* xq,
                                     uint8_t* xs, int32_t* expert_offsets, int32_t* sorted_route,
                                     int32_t* route_row, void* workspace, size_t ws_bytes,
                                     hipStream_t stream);

/* a2 + a3 in one call, for top-k ids and weights computed before the expert
 * layer (page 1 "Serving call chain": the fused MoE call receives the router's
 * top-k ids and weights; its Phase 4 benchmark feeds them in directly).
 * Computes exactly what moe_quant_mxfp8 and then moe_permute compute with the
 * same arguments (same bytes in every output and in the workspace), and
 * accepts what those two accept together (every check of each).  When the
 * grouping runs as one workgroup (T * top_k <= 2048) it is a single launch,
 * workgroup 0 grouping while the others quantise; otherwise it issues the two
 * calls' launches in order on `stream`. */
moe_status_t moe_quant_permute(const uint16_t* x, int64_t ld_x, int T, int H,
                               const int32_t* topk_idx, int top_k, int expert_offset,
                               int E_local, uint8_t* xq, uint8_t* xs, int32_t* expert_offsets,
                               int32_t* sorted_route, int32_t* route_row, void* workspace,
                               size_t ws_bytes, hipStream_t stream);

/* a4 + a5 + a6 -- FC1 grouped GEMM, SiTU, requantisation (page 1 "Serving call
 * chain": grouped GEMM1 then gated activation; "Real checkpoint contract": w13
 * holds [gate; up] in two contiguous halves, SiTU gate' = alpha *
 * tanh(gate/alpha) * sigmoid(gate), up' = beta * tanh(up/beta), out = gate' *
 * up' with alpha = 4, beta = 25; page 5: w13 [E, 2I, H/2], scales
 * [E, 2I, H/32]).
 *   xq, xs          MXFP8 activations from moe_quant_mxfp8 ([T, H], [T, H/32]).
 *   expert_offsets, sorted_route   from moe_permute; grouped row j of expert e
 *                   multiplies token sorted_route[j] / top_k.
 *   w13, w13_s      uint8 [E_local, 2I, H/2], [E_local, 2I, H/32] (local window).
 *   hq, hs          uint8 [T*top_k, I], [T*top_k, I/32]: the SiTU output of
 *                   each kept grouped row, requantised with the moe_quant_mxfp8
 *                   rule from the float accumulators (rows past the kept count
 *                   are not written).
 *   workspace       the buffer moe_permute filled. */
moe_status_t moe_fc1_situ(const uint8_t* xq, const uint8_t* xs, int T, int H, int I, int top_k,
                          int E_local, const int32_t* expert_offsets,
                          const int32_t* sorted_route, const uint8_t* w13,
                          const uint8_t* w13_s, float situ_alpha, float situ_beta,
                          uint8_t* hq, uint8_t* hs, void* workspace, size_t ws_bytes,
                          hipStream_t stream);

/* a7 + a8 -- FC2 grouped GEMM and top-k combine (page 1 "Serving call chain":
 * GEMM2 then finalize; "Phase 2": the non-fused finalize for bitwise
 * determinism, next to the fused atomic one; page 5: w2 [E, H, I/2], scales
 * [E, H, I/32]).
 *   hq, hs          from moe_fc1_situ.
 *   expert_offsets, sorted_route, route_row   from moe_permute.
 *   topk_w          from moe_route (float [T, top_k]).
 *   w2, w2_s        uint8 [E_local, H, I/2], [E_local, H, I/32].
 *   mode            a moe_combine_t value (else MOE_ERR_ENUM).
 *   out             bf16 bits [T, H], row stride ld_out (>= H, multiple of 8):
 *                   out[t] = bf16_rne( sum over kept k of
 *                   topk_w[t,k] * y[route_row[t,k]] ) with float accumulation
 *                   (DETERMINISTIC: in k order, bitwise repeatable; ATOMIC: in
 *                   the order the atomic adds land); a token with no kept slot
 *                   gets zeros.
 *   workspace       the buffer moe_permute filled, of at least
 *                   moe_workspace_size(..., mode) bytes (DETERMINISTIC: holds
 *                   the per-route FC2 rows y [T*top_k, H] as fp16 of y / 2^e
 *                   with one exponent e per 64 columns, 2^-11 relative, below
 *                   the output's bf16 step; ATOMIC: the float [T, H] sums). */
moe_status_t moe_fc2_combine(const uint8_t* hq, const uint8_t* hs, int T, int H, int I,
                             int top_k, int E_local, const int32_t* expert_offsets,
                             const int32_t* sorted_route, const int32_t* route_row,
                             const float* topk_w, const uint8_t* w2, const uint8_t* w2_s,
                             int mode, uint16_t* out, int64_t ld_out, void* workspace,
                             size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Tiled weight layout (optional, one-time).  The calls above read the
 * checkpoint layout directly.  moe_prepack_w13 / moe_prepack_w2 reorder the
 * same bytes once, at load time, into a tiled layout whose blocks the FC
 * kernels read as whole contiguous pieces; moe_fc1_situ_tiled /
 * moe_fc2_combine_tiled then compute exactly what moe_fc1_situ /
 * moe_fc2_combine compute (this is the role of the weight and scale
 * transforms the pages apply after loading, page 5).
 *
 * Tiled layout, for a weight matrix of N rows and K columns per expert
 * (w13: N = 2I, K = H; w2: N = H, K = I): rows are grouped 512 at a time
 * (group cg) and K is cut into stages of 128.  Block (e, cg, s) holds
 *   data   32768 bytes: 16-byte chunk number (4w + i) * 64 + l is the logical
 *          16-byte chunk c = (l & 3) ^ ((l >> 3) & 3) of stage s of row
 *          r = 64w + 16i + l/4 (w < 8, i < 4, l < 64);
 *   scales 2048 bytes: dword r = the four scale bytes of row r for MX blocks
 *          4s .. 4s+3;
 * where group row r is global row: w13 — unit u = 8cg + r/64, b = (r/16) % 4,
 * row = (b < 2 ? 0 : I) + 32u + 16(b % 2) + r % 16 (gate rows of the unit,
 * then the matching up rows); w2 — 512cg + r.  Blocks are stored in
 * [e][cg][s] order; the tiled data and scale arrays have the sizes of the
 * checkpoint arrays.  Requires I % 256 == 0 (w13) and H % 512 == 0 (w2).
 * ------------------------------------------------------------------------- */

/* Reorder checkpoint w13 [E_local, 2I, H/2] + w13_s [E_local, 2I, H/32] into
 * w13t / w13t_s (same sizes, distinct buffers).  Asynchronous on `stream`. */
moe_status_t moe_prepack_w13(const uint8_t* w13, const uint8_t* w13_s, int E_local, int H, int I,
                             uint8_t* w13t, uint8_t* w13t_s, hipStream_t stream);

/* Row order of a w13 tensor (fixed values).  Page 1 ("Real checkpoint
 * contract") lists three: the Kimi-K3 checkpoint keeps [gate; up] halves
 * (rows [0, I) gate, [I, 2I) up), the CUTLASS runner expects [up; gate]
 * halves, and the GPT-OSS loader interleaves rows (row 2j gate j, row 2j+1 up
 * j; page 3's de-interleave takes rows 0::2 as gate, 1::2 as up). */
typedef enum moe_w13_layout {
  MOE_W13_GATE_UP = 0,
  MOE_W13_UP_GATE = 1,
  MOE_W13_INTERLEAVED = 2
} moe_w13_layout_t;

/* moe_prepack_w13 for a w13 / w13_s whose rows are in `layout` order (a
 * moe_w13_layout_t value; anything else is MOE_ERR_ENUM).  The tiled result
 * is the same bytes moe_prepack_w13 gives for the [gate; up] reordering of
 * the input, so moe_fc1_situ_tiled computes the same layer for every layout.
 * (The checkpoint-layout moe_fc1_situ reads [gate; up] only.) */
moe_status_t moe_prepack_w13_layout(const uint8_t* w13, const uint8_t* w13_s, int E_local, int H,
                                    int I, int layout, uint8_t* w13t, uint8_t* w13t_s,
                                    hipStream_t stream);

/* Reorder checkpoint w2 [E_local, H, I/2] + w2_s [E_local, H, I/32]. */
moe_status_t moe_prepack_w2(const uint8_t* w2, const uint8_t* w2_s, int E_local, int H, int I,
                            uint8_t* w2t, uint8_t* w2t_s, hipStream_t stream);

/* moe_fc1_situ on tiled w13 (from moe_prepack_w13); same results. */
moe_status_t moe_fc1_situ_tiled(const uint8_t* xq, const uint8_t* xs, int T, int H, int I,
                                int top_k, int E_local, const int32_t* expert_offsets,
                                const int32_t* sorted_route, const uint8_t* w13t,
                                const uint8_t* w13t_s, float situ_alpha, float situ_beta,
                                uint8_t* hq, uint8_t* hs, void* workspace, size_t ws_bytes,
                                hipStream_t stream);

/* moe_fc2_combine on tiled w2 (from moe_prepack_w2); same results. */
moe_status_t moe_fc2_combine_tiled(const uint8_t* hq, const uint8_t* hs, int T, int H, int I,
                                   int top_k, int E_local, const int32_t* expert_offsets,
                                   const int32_t* sorted_route, const int32_t* route_row,
                                   const float* topk_w, const uint8_t* w2t,
                                   const uint8_t* w2t_s, int mode, uint16_t* out,
                                   int64_t ld_out, void* workspace, size_t ws_bytes,
                                   hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Around the experts: what one MoE block runs between the residual stream and
 * the five calls above (additions to ABI version 3; nothing above changes).
 *
 *   moe_add_rmsnorm   residual addition + RMS norm, bf16 and 8-bit outputs
 *   moe_gate_logits   the router's product, bf16 x bf16 -> float32 logits
 *   moe_route_groups  sigmoid / softmax, group-limited top-k routing
 *   moe_quant_int8, moe_int8_matmul, moe_int8_linear
 *                     dense projections in 8-bit integers (into and out of the
 *                     experts' width), one scale per token and per channel
 *
 * The conventions above hold.  Rows: 0 <= T (M) <= 4194303.
 * ------------------------------------------------------------------------- */

/* The 8-bit output of moe_add_rmsnorm (fixed values). */
typedef enum moe_q8 {
  MOE_Q8_NONE = 0,
  MOE_Q8_MXFP8 = 1,  /* E4M3 + one E8M0 per 32 elements: moe_fc1_situ's xq, xs */
  MOE_Q8_INT8 = 2    /* int8 + one float per row: moe_int8_matmul's xq, xs */
} moe_q8_t;

/* Output type of the 8-bit integer products (fixed values). */
typedef enum moe_out {
  MOE_OUT_BF16 = 0,
  MOE_OUT_F32 = 1
} moe_out_t;

/* Scores of moe_route_groups (fixed values). */
typedef enum moe_score {
  MOE_SCORE_SIGMOID = 0,
  MOE_SCORE_SOFTMAX = 1
} moe_score_t;

/* What a group of experts is worth in moe_route_groups (fixed values). */
typedef enum moe_group_score {
  MOE_GROUP_MAX = 0,   /* its largest key */
  MOE_GROUP_TOP2 = 1   /* the float sum of its two largest keys */
} moe_group_score_t;

/* Residual addition, root-mean-square norm and 8-bit output, in one pass.
 *   h = x + residual in float (x alone without one), y = (h * weight) *
 *   (1 / sqrt(mean(h^2) + eps)) in float, each output rounded once from there:
 *   residual_out  bf16(h), or NULL for none; may be x or residual itself (the
 *                 same pointer and stride), for an update in place.
 *   y             bf16(y), or NULL for none (at least one of y and xq); may be
 *                 x itself.  Other overlaps of outputs and inputs are not
 *                 allowed.
 *   q8            a moe_q8_t value.  MXFP8: xq uint8 [T, H], xs uint8
 *                 [T, H/32], the rule of moe_quant_mxfp8 applied to the float
 *                 y (H a multiple of 32).  INT8: xq int8 [T, H], xs float [T],
 *                 the rule of moe_quant_int8 applied to the float y.  NONE: xq
 *                 and xs are not used.
 *   x, residual   bf16 bits [T, H], row strides ld_x, ld_residual; residual
 *                 may be NULL.  weight: bf16 bits [H].  eps >= 0, finite.
 *   H a multiple of 8, at most 32768; row strides >= H and multiples of 8.
 *   A row whose squares overflow float, or that holds an infinity or a NaN,
 *   gives what these formulas give (zeros and NaN). */
moe_status_t moe_add_rmsnorm(const uint16_t* x, int64_t ld_x, const uint16_t* residual,
                             int64_t ld_residual, const uint16_t* weight, float eps, int T,
                             int H, int q8, uint16_t* residual_out, int64_t ld_residual_out,
                             uint16_t* y, int64_t ld_y, void* xq, void* xs,
                             hipStream_t stream);

/* Rows in 8-bit integers, one scale per row: s = max(absmax / 127, 2^-126),
 * q = clamp(rint(x * (1 / s)), -127, 127), ties to even, all in float.  A row
 * holding an infinity or a NaN gets s = NaN and q = 0, so that its products
 * are NaN.  Tokens (one scale per token) and, at load time, weight rows (one
 * scale per output channel) alike.
 *   x  bf16 bits [T, H], row stride ld_x (>= H, multiple of 8); H a multiple
 *   of 8, at most 32768.   xq  int8 [T, H] (8-byte aligned rows); xs  float [T]. */
moe_status_t moe_quant_int8(const uint16_t* x, int64_t ld_x, int T, int H, int8_t* xq,
                            float* xs, hipStream_t stream);

/* Bytes of workspace for moe_int8_linear (and so for moe_int8_matmul) with
 * these sizes: the product's partial sums, and the tokens in 8 bits with their
 * scales.  It grows with M, so a buffer for M rows serves every smaller M with
 * the same N and K.  0 for invalid sizes. */
size_t moe_int8_workspace_size(int M, int N, int K);

/* Bytes of workspace for moe_int8_matmul alone, whose tokens are in 8 bits
 * already: the partial sums, at most 16 MB.  It grows with M.  0 for M = 0 and
 * for invalid sizes. */
size_t moe_int8_matmul_workspace_size(int M, int N, int K);

/* out[m, n] = (sum_k xq[m, k] * w[n, k]) * xs[m] * w_s[n]: the sum exact in
 * int32, the three factors multiplied in float in this order, one rounding to
 * out_type.
 *   xq   int8 [M, K], row stride ld_xq (>= K, multiple of 16); xs float [M].
 *   w    int8 [N, K]; w_s float [N].
 *   out  [M, N] of out_type (a moe_out_t value), row stride ld_out >= N; 16-byte
 *        aligned (bf16) or 4-byte aligned (float); vector stores where ld_out
 *        is a multiple of 4 and out is 16-byte aligned.
 *   K a multiple of 16, 16 <= K <= 131056 (no int32 overflow); 1 <= N <= 2^20.
 *   workspace  at least moe_int8_matmul_workspace_size bytes, 256-byte aligned. */
moe_status_t moe_int8_matmul(const int8_t* xq, int64_t ld_xq, const float* xs, const int8_t* w,
                             const float* w_s, int M, int N, int K, int out_type, void* out,
                             int64_t ld_out, void* workspace, size_t ws_bytes,
                             hipStream_t stream);

/* moe_quant_int8 of x [M, K] (bf16 bits, row stride ld_x), then
 * moe_int8_matmul of the result (kept in the workspace, which has at least
 * moe_int8_workspace_size bytes): same output.  K at most 32768. */
moe_status_t moe_int8_linear(const uint16_t* x, int64_t ld_x, const int8_t* w, const float* w_s,
                             int M, int N, int K, int out_type, void* out, int64_t ld_out,
                             void* workspace, size_t ws_bytes, hipStream_t stream);

/* Bytes of workspace for moe_gate_logits; it grows with T.  0 for T = 0 and
 * for invalid sizes. */
size_t moe_gate_workspace_size(int T, int E, int H);

/* The router's product: logits[t, e] = sum_h x[t, h] * w[e, h], products of
 * bf16 values summed in float (the order is fixed for given sizes and row
 * strides).
 *   x  bf16 bits [T, H], row stride ld_x (>= H, multiple of 8); w bf16 bits
 *   [E, H]; logits float [T, E], row stride ld_logits >= E.
 *   1 <= E <= 4096; H a multiple of 8, 8 <= H <= 1048576. */
moe_status_t moe_gate_logits(const uint16_t* x, int64_t ld_x, const uint16_t* w, int T, int E,
                             int H, float* logits, int64_t ld_logits, void* workspace,
                             size_t ws_bytes, hipStream_t stream);

/* Routing with groups of experts.
 *   score: s_e = sigmoid(l_e), or exp(l_e - max) / sum over the experts that
 *   their logits do not mask, evaluated in double and rounded once to float.
 *   key_e = s_e + bias_e in float (bias NULL: s_e).  An expert is masked for a
 *   token when its logit is -inf or the lowest finite float, or its key is
 *   -inf.  The bias takes part in the choice only: an expert whose bias is -inf
 *   is never taken but keeps its share of the softmax, so that the weights of
 *   the others do not depend on biases (without renormalise they then add up to
 *   less than without that expert).
 *   The experts stand in n_group groups of E / n_group neighbours; the
 *   topk_group groups of most worth (group_score; masked experts do not count)
 *   stay, and of their experts the top_k with the largest keys, in descending
 *   order.  Equal worths and equal keys rank the lower index first; NaN ranks
 *   below every number.  A group of masked experts only ranks last.
 *   w_k = s_k, divided by sum_j s_j (double, left to right; 0 where that sum
 *   is 0) if renormalise is not 0, times routed_scaling, rounded to float.
 *   Slots for which no unmasked expert is left hold id -1 and weight 0 (the
 *   masked slots of moe_permute); a token whose experts are all masked gets
 *   only those.
 *   topk_idx int32 [T, top_k], topk_w float [T, top_k].
 *   With one group, sigmoid, renormalise and no masked expert the results are
 *   those of moe_route.
 *   1 <= top_k <= min(64, topk_group * (E / n_group)); 1 <= topk_group <=
 *   n_group <= 64; E a multiple of n_group, at most 4096.
 *   Speed: with n_group rounded up to a power of two, groups of up to 1024 /
 *   n_group experts (1024 experts in one group, 8 groups of 128, but 9 groups
 *   of 64) have their choice narrowed in float; for larger ones every score is
 *   evaluated in double, in 2 to 8 times the time per expert. */
moe_status_t moe_route_groups(const float* logits, int64_t ld_logits, const float* bias, int T,
                              int E, int top_k, int n_group, int topk_group, int score,
                              int group_score, int renormalise, float routed_scaling,
                              int32_t* topk_idx, float* topk_w, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Products in 8-bit floating point with a scale for each block of 128 (the
 * format of checkpoints that store E4M3 weights beside one float per block of
 * 128 x 128).  Additions to ABI version 3; the conventions above hold.
 *
 *   moe_quant_fp8    bf16 tokens -> E4M3, one float per token and 128 elements
 *   moe_fp8_matmul, moe_fp8_linear    dense, from E4M3 and from bf16 tokens
 *   moe_fp8_grouped  the rows of every expert times that expert's weight
 *
 * Blocks: KB = ceil(K / 128) along the contraction, NB = ceil(N / 128) along
 * the weight's rows; the last block of either may be shorter.
 *   xq   E4M3 [M, K], row stride ld_xq (>= K, a multiple of 16).
 *   xs   float [KB, M], row stride ld_xs (>= M): the scale of token m's block b
 *        is xs[b, m] (tokens side by side: the products read one block of many
 *        tokens at a time).
 *   w    E4M3 [N, K]; w_s float [NB, KB]; experts one after another.
 *   out  bf16 [M, N], row stride ld_out (>= N, any), 16-byte aligned.
 *   out[m, n] = sum_b (xs[b, m] * w_s[n / 128, b]) * (sum_{k in b} xq[m, k] w[n, k])
 *   rounded once to bf16; the scales' product and the sum over blocks in float,
 *   the sum within a block by the matrix unit, whose accumulation keeps about
 *   17 bits of that block's sum of |products|: below the output's 8.  The order
 *   of the sum is fixed for given sizes and row strides.  Codes 0x7F and 0xFF
 *   are NaN.
 *   With the weight transposed (w as [K, N], w_s as [KB, NB]) the same calls
 *   give the gradient with respect to the tokens: dx = dout . w.
 *   Tokens of which 256 rows span 2 GiB (256 * ld_xq + K), and scales that do (4 *
 *   KB * ld_xs), take the kernel of few tokens at any M, which is far slower.
 *   K a multiple of 16, 16 <= K <= 2^20; 1 <= N <= 2^20; 0 <= M <= 4194303.
 * ------------------------------------------------------------------------- */

/* xs[b, t] = max(absmax of the block / 448, 2^-126), xq = E4M3 of x * (1 / xs),
 * nearest, ties to even, in float.  A block that holds an infinity or a NaN
 * gets the scale NaN and codes 0, so that the token's products are NaN.
 *   x  bf16 bits [T, H], row stride ld_x (>= H, multiple of 8); H as K above.
 *   xq uint8 [T, H]; xs float [ceil(H / 128), T], row stride ld_xs.
 *   More tokens than a call takes are quantised in pieces: tokens [t0, t0 + T) of
 *   a larger xs are xs + t0 with that one's ld_xs. */
moe_status_t moe_quant_fp8(const uint16_t* x, int64_t ld_x, int T, int H, uint8_t* xq, float* xs,
                           int64_t ld_xs, hipStream_t stream);

/* Bytes of workspace for moe_fp8_linear (and so for moe_fp8_matmul) with these
 * sizes: the product's partial sums, and the tokens in 8 bits with their
 * scales.  It grows with M, so a buffer for M rows serves every smaller M with
 * the same N and K.  0 for invalid sizes. */
size_t moe_fp8_workspace_size(int M, int N, int K);

/* Bytes of workspace for moe_fp8_matmul alone: the partial sums, at most
 * 16 MB.  It grows with M (so products of many rows, which are not split, name
 * it as well).  0 for up to 8 rows and for K up to 640, which are never split,
 * and for invalid sizes; workspace may be NULL then. */
size_t moe_fp8_matmul_workspace_size(int M, int N, int K);

moe_status_t moe_fp8_matmul(const uint8_t* xq, int64_t ld_xq, const float* xs, int64_t ld_xs,
                            const uint8_t* w, const float* w_s, int M, int N, int K, uint16_t* out,
                            int64_t ld_out, void* workspace, size_t ws_bytes, hipStream_t stream);

/* moe_quant_fp8 of x [M, K] (bf16 bits, row stride ld_x, a multiple of 8) and
 * moe_fp8_matmul as one call. */
moe_status_t moe_fp8_linear(const uint16_t* x, int64_t ld_x, const uint8_t* w, const float* w_s,
                            int M, int N, int K, uint16_t* out, int64_t ld_out, void* workspace,
                            size_t ws_bytes, hipStream_t stream);

/* Rows in expert order times their expert's weight: for expert e and output row
 * j of [expert_offsets[e], expert_offsets[e + 1]),
 *   out[j] = token(j) . w[e]^T,  token(j) = sorted_route[j] / top_k, or j itself
 *   where sorted_route is NULL (tokens that stand in expert order already).
 *   xq [rows, K], xs [KB, rows]; w [E_local, N, K], w_s [E_local, NB, KB];
 *   expert_offsets int32 [E_local + 1] and sorted_route int32 [R] as moe_permute
 *   gives them (read on the GPU: the call does not synchronise); out [R, N].
 *   Output rows before the first offset and behind the last are left as they
 *   were; offsets past R and routes past the tokens' rows are cut off there.
 *   Offsets do not descend.  Where they do, an expert whose end is before its
 *   start has no rows, and the experts' rows may come to more tiles than R has:
 *   then a row that any expert claims, one or several, holds, element by element,
 *   a claimant's values or what was there.  Other rows are left as they were.
 *   Tokens read through sorted_route that span 2 GiB or more (rows * ld_xq + K),
 *   256 rows that span as much without it, and scales that do (4 * KB * ld_xs) take
 *   a simpler kernel, several times slower: many tokens are better put into expert
 *   order first (moe_sort_tokens).
 *   1 <= E_local <= 4096; 0 <= rows, R <= 2^30; without sorted_route rows >= R. */
moe_status_t moe_fp8_grouped(const uint8_t* xq, int64_t ld_xq, const float* xs, int64_t ld_xs,
                             int rows, const uint8_t* w, const float* w_s, int E_local, int N,
                             int K, const int32_t* expert_offsets, const int32_t* sorted_route,
                             int top_k, int R, uint16_t* out, int64_t ld_out,
                             hipStream_t stream);

/* ---------------------------------------------------------------------------
 * Tokens into expert order and back, and the gradients, for experts that run
 * outside the five calls and for their training.  route_row int32 [T, top_k] as
 * moe_permute gives it; a route whose row is negative or not below n_rows has
 * no part.  Rows may have any length and stride and start at any element; sums
 * in float, in slot order, one rounding; equal calls give equal bits.  (A row
 * that several routes name, as moe_permute's never do, gets, element by element,
 * what one of them brings.)
 * 1 <= H <= 2^20; 1 <= top_k <= 64; T * top_k <= 2^30; 0 <= n_rows <= 2^30
 * (T * top_k serves every routing; fewer where the caller knows that no more
 * routes are kept).
 * ------------------------------------------------------------------------- */

/* Element type of the rows (fixed values). */
typedef enum moe_rows {
  MOE_ROWS_BF16 = 0,
  MOE_ROWS_F32 = 1
} moe_rows_t;

/* rows[route_row[t, k]] = x[t] for every kept route; other rows are left as
 * they were.  Its gradient is moe_unsort_tokens without weights.
 *   x [T, H], row stride ld_x; rows [n_rows, H], row stride ld_rows; no overlap. */
moe_status_t moe_sort_tokens(const void* x, int64_t ld_x, int T, int H, int top_k,
                             const int32_t* route_row, int type, void* rows, int64_t ld_rows,
                             int n_rows, hipStream_t stream);

/* out[t] = sum over kept k of topk_w[t, k] * rows[route_row[t, k]]; with topk_w
 * NULL the plain sum.  A token with no kept route gets zeros.
 *   rows [n_rows, H], row stride ld_rows; topk_w float [T, top_k]; out [T, H],
 *   row stride ld_out; no overlap. */
moe_status_t moe_unsort_tokens(const void* rows, int64_t ld_rows, int n_rows, int T, int H,
                               int top_k, const int32_t* route_row, const float* topk_w, int type,
                               void* out, int64_t ld_out, hipStream_t stream);

/* Gradients of the weighted moe_unsort_tokens:
 *   drows[route_row[t, k]] = topk_w[t, k] * dout[t] (other rows left as they were),
 *   dw[t, k] = sum_h dout[t, h] * rows[route_row[t, k], h] in float (0 for a
 *   route that is not kept).
 *   drows [n_rows, H], row stride ld_drows, or NULL for none; dw float [T,
 *   top_k], or NULL for none (rows is not read then); at least one of the two;
 *   no overlap. */
moe_status_t moe_unsort_tokens_grad(const void* dout, int64_t ld_dout, const void* rows,
                                    int64_t ld_rows, int n_rows, int T, int H, int top_k,
                                    const int32_t* route_row, const float* topk_w, int type,
                                    void* drows, int64_t ld_drows, float* dw, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MI355MOE_H */
