// kernels.hpp -- host-side launchers of the gfx950 kernels (internal to libmoe).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

struct FfnArgs;

hipError_t launch_topk(const float* logits, int T, int E, int k, int32_t* ids, float* w, hipStream_t st);
// Router projection: logits [T][E] = x [T][H] . wr [E][H]^T (bf16 in, f32 out).
hipError_t launch_router_logits(const uint16_t* x, const uint16_t* wr, int T, int H, int E, float* logits,
                                hipStream_t st);
// Top-k then permutation; one workgroup launch for small batches.
hipError_t launch_route(const float* logits, int T, int E, int k, int32_t* ids, float* w, int32_t* counts,
                        int32_t* offsets, int32_t* sorted_rows, int32_t* inv_rows, hipStream_t st);
hipError_t launch_permute(const int32_t* ids, int T, int k, int E, int32_t* counts, int32_t* offsets,
                          int32_t* sorted_rows, int32_t* inv_rows, hipStream_t st);
hipError_t launch_combine(const float* rows, const float* w, const int32_t* inv, const float* shared, int T, int k,
                          int H, void* y, bool bf16_out, hipStream_t st);

// Elastic cache resize: copy `bytes` of each of n experts from slot from[i] of
// one pool to slot to[i] of another (batched launches, the table in the kernel
// arguments).  Expert bytes must be a multiple of 16 and the pools 16-byte aligned.
constexpr int kMoveBatch = 480;
// The slot tables of one cache wave from up to kSlotPairsMax (expert, slot) pairs
// passed by value: table_a (and table_b if non-null) [E] set to -1, then
// key = expert | (table << 16) (table 0: a, 1: b) gets slot.  E <= 65535.
constexpr int kSlotPairsMax = 240;
struct SlotPairs {
  int32_t* table_a;
  int32_t* table_b;
  int E, n;
  int32_t key[kSlotPairsMax];
  int32_t slot[kSlotPairsMax];
};
hipError_t launch_write_slot_tables(const SlotPairs& p, hipStream_t st);
hipError_t launch_move_slots(const uint8_t* src, uint64_t src_stride, uint8_t* dst, uint64_t dst_stride,
                             uint64_t bytes, const int32_t* from, const int32_t* to, int n, hipStream_t st);

// Grouped FFN phases.  wtype: 0 f32, 1 bf16, 2 mxfp4 (3, MXFP4 with MXFP8
// activations, runs the grouped GEMM only).
hipError_t launch_ffn_gate_up(int wtype, const FfnArgs& a, hipStream_t st);
hipError_t launch_ffn_down(int wtype, const FfnArgs& a, hipStream_t st);
// Prefill-sized batches (LDS-staged token tiles); same arguments and results.
bool prefill_supported(int wtype, int H, int I, int I_shared);
hipError_t launch_prefill_gate_up(int wtype, const FfnArgs& a, hipStream_t st);
hipError_t launch_prefill_down(int wtype, const FfnArgs& a, hipStream_t st);
// Native FP4 path: MXFP8 activations (E4M3 codes [T][H], E8M0 scales [T][H/32])
// from bf16 x, then gate_up on the scaled f8f6f4 MFMA (a.xq, a.xs); the down phase
// is launch_prefill_down with MXFP4 weights.
hipError_t launch_mx8_quantize(const uint16_t* x, int T, int H, uint8_t* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_native_gate_up(const FfnArgs& a, hipStream_t st);
// Workspace bytes: the SwiGLU intermediate for T*k routed + T shared rows; for the
// native path (wtype 3) also the MXFP8 activations, at ffn_workspace_xq_offset.
size_t ffn_workspace_bytes(int wtype, int T, int k, int H, int I, int I_shared);
size_t ffn_workspace_xq_offset(int T, int k, int I, int I_shared);

// One layer for a few tokens in two kernels (decode_layer.hip).  wtype: 1 bf16, 2 mxfp4.
constexpr int kDecodeLayerMaxT = 64, kDecodeLayerMaxPairs = 512;
struct DecodeLayerArgs {
  const uint8_t* slot_pool;
  uint64_t slot_stride;
  const int32_t* slot_of_expert;  // [E], -1: the expert contributes nothing
  const uint8_t* shared_w;        // nullable
  const uint16_t* x;              // [T][H] bf16
  const float* logits;            // [T][E], or null: ids and w are given
  int32_t* ids;                   // [T][k]
  float* w;                       // [T][k]
  uint16_t* h;                    // workspace: [T*k + T][2][h_ld] bf16 (h and the remainder of its rounding)
  void* plan;                     // workspace: decode_layer_plan_bytes()
  void* y;                        // [T][H]
  int T, k, E, H, I, I_shared, h_ld;
};
size_t decode_layer_plan_bytes();
constexpr int kDecodeLayerMaxH = 65536;  // one token row fits the gate/up kernel's LDS
hipError_t launch_decode_layer(int wtype, const DecodeLayerArgs& a, bool bf16_out, hipStream_t st);

// Linear product with 4-bit weights (w4.hip).  fmt: W_MXFP4 or W_INT4.
struct W4Args {
  const uint8_t* w;    // laid out by launch_w4_pack
  const uint16_t* x;   // rows of K bf16, x_ld elements apart
  const float* bias;   // [N] or null
  void* y;             // rows of N, y_ld elements apart
  int64_t x_ld, y_ld;
  int T, N, K, group;
};
// Bytes of the laid-out matrix.
size_t w4_bytes(int fmt, int N, int K, int group);
hipError_t launch_w4_pack(int fmt, const uint8_t* codes, const void* scales, const uint8_t* zeros, int N, int K,
                          int group, uint8_t* w, hipStream_t st);
hipError_t launch_w4_linear(int fmt, const W4Args& a, bool bf16_out, hipStream_t st);

// The boundary of two blocks (block_norm.hip).
enum NormKind { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
struct BlockNormArgs {
  const void* block;  // nullable
  const float* post_w;
  const float* post_b;
  const void* gate;  // nullable; rows gate_ld apart (0: one row for every token)
  const void* res;   // nullable
  const float* pre_w;
  const float* pre_b;
  void* res_out;  // nullable
  void* x;        // nullable
  int64_t b_ld, gate_ld, r_ld, ro_ld, x_ld;
  float block_scale, res_scale, eps;
  int T, H, post_kind, pre_kind;
  bool gate_bf16;
};
constexpr int kBlockNormMaxH = 32768;  // a row in the registers of 1024 threads, 32 elements each
hipError_t launch_block_norm(const BlockNormArgs& a, bool block_bf16, bool res_bf16, bool x_bf16, hipStream_t st);

// Linear product with bias, activation and residual (linear.hip); f32 or bf16 operands.
enum Activation { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };
struct LinearArgs {
  const void* w;      // N rows of K, w_ld elements apart
  const void* x;      // T rows of K, x_ld elements apart
  const float* bias;  // [N] or null
  const void* res;    // T rows of N, r_ld elements apart, or null
  void* y;            // T rows of N, y_ld elements apart
  int64_t w_ld, x_ld, r_ld, y_ld;
  int T, N, K, act;
  bool res_bf16, y_bf16;
};
int linear_tile(bool bf16, int T, int N, int K);  // of the kernel that launch_linear takes: weight rows << 16 | tokens
hipError_t launch_linear(bool bf16, const LinearArgs& a, hipStream_t st);

// Tokens sorted by expert and back, with the gradients (token_sort.hip).
struct DispatchArgs {
  const void* x;  // T rows of H, x_ld elements apart
  const int32_t* ids;
  int32_t* counts;
  int32_t* offsets;
  int32_t* sorted_rows;
  int32_t* inv_rows;
  void* rows;  // n_rows rows of H, rows_ld elements apart
  int64_t x_ld, rows_ld;
  int T, k, E, H, n_rows;
  bool pass;  // set by the launcher: rows are written past the caches
};
size_t dispatch_workspace_bytes(int T, int k, int E);
hipError_t launch_dispatch(DispatchArgs a, int32_t* table, bool bf16, hipStream_t st);
struct CombineRowsArgs {
  const void* rows;       // n_rows rows of H, rows_ld elements apart
  const float* topk_w;    // [T][k]; the forward sum: null for weights of 1
  const int32_t* inv_rows;
  void* y;                // T rows of H, y_ld elements apart (backward: dy, read)
  void* d_rows;           // backward: n_rows rows of H, dr_ld elements apart
  float* d_w;             // backward: [T][k]
  int64_t rows_ld, y_ld, dr_ld;
  int T, k, H, n_rows;
  bool pass;              // backward, set by the launcher: d_rows are written past the caches
};
hipError_t launch_combine_rows(const CombineRowsArgs& a, bool rows_bf16, bool y_bf16, hipStream_t st);
hipError_t launch_combine_rows_backward(CombineRowsArgs a, bool dy_bf16, bool rows_bf16, hipStream_t st);
hipError_t launch_gate_backward(const int32_t* ids, const float* w, const float* d_w, int T, int E, int k,
                                float* d_logits, hipStream_t st);

}  // namespace moe
