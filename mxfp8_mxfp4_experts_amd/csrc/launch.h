// Kernel launchers behind the C ABI (arguments already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mi355moe.h"

namespace mi355moe {

hipError_t launch_route(const float* logits, int64_t ld, const float* bias, int T, int E, int K,
                        float scaling, int32_t* idx, float* w, hipStream_t stream);
hipError_t launch_quant(const uint16_t* x, int64_t ld, int T, int H, uint8_t* xq, uint8_t* xs,
                        hipStream_t stream);
// counts: int32 [perm_chunks(R)][E_local] scratch (used when R > kPermSingle).
hipError_t launch_permute(const int32_t* idx, int R, int offset, int E_local, int32_t* offs,
                          int32_t* sorted_route, int32_t* route_row, int32_t* tile_prefix,
                          int32_t* counts, hipStream_t stream);
// Route + quantise + group in one launch (front.hip), for batches that
// front_fusable accepts (T <= 16, E <= 1024, its LDS within 64 KB); the same
// bytes as launch_route, launch_quant and launch_permute.
bool front_fusable(int T, int E, int K, int E_local);
hipError_t launch_front(const float* logits, int64_t ld, const float* bias, int T, int E, int K,
                        float scaling, int32_t* topk_idx, float* topk_w, const uint16_t* x,
                        int64_t ld_x, int H, uint8_t* xq, uint8_t* xs, int offset, int E_local,
                        int32_t* offs, int32_t* sorted_route, int32_t* route_row,
                        int32_t* tile_prefix, hipStream_t stream);
// Quantise + group in one launch (front.hip), when the grouping is one
// workgroup (R <= kPermSingle); the same bytes as launch_quant and
// launch_permute.
bool quant_permute_fusable(int64_t R);
hipError_t launch_quant_permute(const uint16_t* x, int64_t ld_x, int T, int H, uint8_t* xq,
                                uint8_t* xs, const int32_t* idx, int R, int offset, int E_local,
                                int32_t* offs, int32_t* sorted_route, int32_t* route_row,
                                int32_t* tile_prefix, hipStream_t stream);
hipError_t launch_fc1(const uint8_t* xq, const uint8_t* xs, int T, int H, int I, int top_k,
                      int E_local, const int32_t* offs, const int32_t* sorted_route,
                      const uint8_t* w13, const uint8_t* w13_s, float alpha, float beta,
                      uint8_t* hq, uint8_t* hs, const int32_t* tile_prefix_all,
                      uint32_t* act_st, int32_t* sched, int n_cu, bool tiled,
                      hipStream_t stream);
// FC2 rows into y / ye (deterministic combine), or, with out_acc set, the
// atomic combine: each grouped row r adds topk_w[route] times its row into
// out_acc [T, H] (route = sorted_route[r]).
hipError_t launch_fc2(const uint8_t* hq, const uint8_t* hs, int T, int H, int I, int top_k,
                      int E_local, const int32_t* offs, const uint8_t* w2, const uint8_t* w2_s,
                      uint16_t* y, int8_t* ye, const int32_t* sorted_route,
                      const float* topk_w, float* out_acc, const int32_t* tile_prefix_all,
                      uint32_t* act_st, int32_t* sched, int n_cu, bool tiled,
                      hipStream_t stream);
struct FcParams;
// Prefill-shaped FC kernels (fc_prefill.hip): usable when K % 128 == 0, the
// weight rows split into whole 512-row groups and the operands fit 32-bit
// buffer offsets.  They read the 256-row tile prefix, and first restage the
// input's scale dwords into prm.act_st (stage-major, grouped-row order).
bool prefill_shape_ok(const FcParams& prm, bool fc1);
hipError_t launch_fc_prefill(bool fc1, bool tiled, FcParams prm, const int32_t* tile_prefix_all,
                             int n_cu, hipStream_t stream);
// One-time reordering of checkpoint-layout weights into the tiled layout
// (layout: w13 row order, 0 [gate; up], 1 [up; gate], 2 interleaved).
hipError_t launch_prepack(bool fc1, const uint8_t* w, const uint8_t* ws, int E_local, int N,
                          int K, int I, int layout, uint8_t* tw, uint8_t* tws,
                          hipStream_t stream);
hipError_t launch_combine(const uint16_t* y, const int8_t* ye, int H, const int32_t* route_row,
                          const float* topk_w, int T, int K, uint16_t* out, int64_t ld_out,
                          hipStream_t stream);
// Atomic combine: clear the float [T, H] sums before FC2; round them to bf16
// after it.
hipError_t launch_acc_clear(float* acc, int T, int H, hipStream_t stream);
hipError_t launch_acc_to_bf16(const float* acc, int T, int H, uint16_t* out, int64_t ld_out,
                              hipStream_t stream);

// Around the experts.
// Residual addition + RMS norm + 8-bit output (norm.hip); norm false: the
// INT8 quantisation of x alone.
struct NormParams {
  const uint16_t* x;
  int64_t ld_x;
  const uint16_t* res;      // may be null
  int64_t ld_res;
  const uint16_t* weight;
  float eps;
  int T, H;
  uint16_t* h;              // may be null
  int64_t ld_h;
  uint16_t* y;              // may be null
  int64_t ld_y;
  uint8_t* xq;
  int64_t ld_q;
  uint8_t* xs;              // E8M0 bytes (MXFP8) or floats (INT8)
};
hipError_t launch_norm(const NormParams& p, int q8, bool norm, hipStream_t stream);

// Group-limited routing (route_groups.hip).
struct RouteGroupsParams {
  const float* logits;
  int64_t ld;
  const float* bias;        // may be null
  int T, E, K, n_group, topk_group, score, group_score, renormalise;
  float scaling;
  int32_t* topk_idx;
  float* topk_w;
};
hipError_t launch_route_groups(const RouteGroupsParams& p, hipStream_t stream);

// Dense products (dense.hip): operands as bytes along K.
struct DenseParams {
  const uint8_t* a;         // [M, Kb], row stride ld_a bytes
  int64_t ld_a;
  const uint8_t* b;         // [N, Kb], row stride ld_b bytes
  int64_t ld_b;
  int M, N, Kb;
  const float* sx;          // INT8: [M], [N] scales
  const float* sw;
  void* out;
  int64_t ld_out;           // elements
  int out_f32;
  int out_vec;              // rows take 4-element vector stores
  void* partial;            // dense_workspace bytes
};
size_t dense_workspace(int M, int N);   // grows with M
// INT8 with bf16 tokens x in one launch (p.a and p.sx unused): the results of
// launch_norm's INT8 quantisation and launch_dense.  dense_fused_q: its Q for
// these sizes, or 0 where the two launches are to be taken.
int dense_fused_q(int M, int N, int K);
hipError_t launch_dense_quant(int q, const DenseParams& p, const uint16_t* x,
                              int64_t ld_x, hipStream_t stream);
hipError_t launch_dense(bool i8, const DenseParams& p, hipStream_t stream);

// Block-scaled FP8 products (fp8.hip).
struct Fp8Params {
  const uint8_t* a;         // tokens [a_rows, K], row stride ld_a
  int64_t ld_a;
  const float* sa;          // their scales [K / 128][a_rows], row stride ld_sa
  int64_t ld_sa;
  const uint8_t* b;         // weights [N, K] or [E, N, K]
  const float* sb;          // their scales [N / 128, K / 128] or [E, ...]
  int M, N, K;              // M: rows of out
  uint16_t* out;
  int64_t ld_out;
  void* partial;            // dense: fp8_workspace bytes
  // Grouped (offs null: dense).
  int E;
  const int32_t* offs;      // [E + 1]
  const int32_t* route;     // [M] or null: output row's token is route / top_k
  int top_k;
  int a_rows;
};
size_t fp8_workspace(int M, int N, int K);   // grows with M
hipError_t launch_quant_fp8(const uint16_t* x, int64_t ld_x, int T, int H, uint8_t* xq,
                            int64_t ld_q, float* xs, int64_t ld_s, hipStream_t stream);
hipError_t launch_fp8(const Fp8Params& p, hipStream_t stream);
// bf16 tokens x in one launch (p.a and p.sa unused), codes made in the product: fp8_raw_q is its Q
// for these sizes, or 0 where quantisation and product are to be two launches.
int fp8_raw_q(int M, int N, int K);
hipError_t launch_fp8_raw(int q, const Fp8Params& p, const uint16_t* x, int64_t ld_x,
                          hipStream_t stream);

// Tokens into expert order and back (sort.hip).
enum class SortOp { kSort, kUnsort, kGrad };
struct SortParams {
  void* x;                  // sort: x; unsort: out; [T, H]
  int64_t ld_x;
  int T, H, top_k;
  const int32_t* route_row; // [T, top_k]
  void* rows;               // [n_rows, H]
  int64_t ld_rows;
  int n_rows;
  const float* w;           // [T, top_k]; unsort: or null
  const void* dout;         // grad: [T, H]
  int64_t ld_dout;
  void* drows;              // grad: or null
  int64_t ld_drows;
  float* dw;                // grad: or null
};
hipError_t launch_sort(const SortParams& p, SortOp op, bool f32, hipStream_t stream);

}  // namespace mi355moe
