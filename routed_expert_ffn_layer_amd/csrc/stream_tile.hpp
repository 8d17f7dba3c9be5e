// stream_tile.hpp -- device pieces of the few-token kernels (the one-call layer and the
// 4-bit linear product): 16 weight rows times up to 16 tokens on
// v_mfma_f32_16x16x32_bf16, weights as the B operand.
//
// Lane l holds weight row l % 16 and k group g = l / 16.  Token i of a tile is row
// 4 * (i % 4) + i / 4 of the A operand, so in the 16 x 16 result lane l holds weight
// row l % 16 and, in element v, token l / 16 + 4 v: up to 4 tokens need element 0
// only, up to 8 elements 0 and 1.  A lane's scale and zero (one row of W) apply to
// its own elements, and the 64 lanes of element v are 4 tokens x 16 rows in order.
#pragma once

#include "ffn_common.hpp"

namespace moe {

// Token of the tile that a lane supplies to the A operand.
__device__ __forceinline__ int a_token(int lane) {
  const int r = lane & 15;
  return (r >> 2) + 4 * (r & 3);
}

// An offset past the end of every buffer read here (all under 2 GiB - 16): the load
// returns zeros.
constexpr int kPastEnd = 0x7ffffff0;

// Byte offset, inside a token row, of fragment m of step s for k group g, or kPastEnd
// past column K (K a multiple of 32).  MXFP4 follows the slot layout (a lane owns a whole
// 32-element block), words of other 4-bit codes hold 8 columns of block m.
template <int FMT>
__device__ __forceinline__ int frag_offset(int s, int m, int g, int K) {
  if constexpr (FMT == W_MXFP4) return s * 128 + 32 * g < K ? s * 256 + 64 * g + 16 * m : kPastEnd;
  return s * 128 + 32 * m < K ? s * 256 + 64 * m + 16 * g : kPastEnd;
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), b, c, 0, 0, 0);
}

}  // namespace moe
