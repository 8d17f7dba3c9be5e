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

// Token fragments of a step: bf16 has one 32-wide MFMA per step, the 4-bit types four.
template <int WT>
struct StepFrags {
  static constexpr int value = WT == W_BF16 ? 1 : 4;
};

// Byte offset, inside a token row, of fragment m of step s for k group g, or kPastEnd
// past column K (K a multiple of 32).  bf16 and MXFP4 follow the slot layout (an MXFP4
// lane owns a whole 32-element block); INT4 words hold 8 columns of block m.
template <int WT>
__device__ __forceinline__ int frag_offset(int s, int m, int g, int K) {
  if constexpr (WT == W_BF16) return s * 64 + 16 * g;
  if constexpr (WT == W_MXFP4) return s * 128 + 32 * g < K ? s * 256 + 64 * g + 16 * m : kPastEnd;
  return s * 128 + 32 * m < K ? s * 256 + 64 * m + 16 * g : kPastEnd;
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), b, c, 0, 0, 0);
}

// One chunk of up to U steps in registers: weight fragments, MXFP4 scale words and the
// token fragments of one token tile.
template <int WT, int U>
struct StreamChunk {
  u32x4 w[U];
  uint32_t sc[U];
  u32x4 x[U][StepFrags<WT>::value];
};

// Steps s .. s+U-1 of row tile `tile` (steps past s1 - 1 re-read it and are not used).
// row_off: byte offset of this lane's token row in xbuf.
template <int WT, int U>
__device__ __forceinline__ void stream_load(StreamChunk<WT, U>& c, const Mat& w, int tile, int s, int s1,
                                            __amdgpu_buffer_rsrc_t xbuf, int row_off) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int su = min(s + u, s1 - 1);
    c.w[u] = bld16(w.codes, lane * 16, (tile * w.nK + su) * 1024);
    if constexpr (WT == W_MXFP4) c.sc[u] = load_scale_word(w, lane, tile, su);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int su = min(s + u, s1 - 1);
#pragma unroll
    for (int m = 0; m < StepFrags<WT>::value; ++m) {
      const int o = frag_offset<WT>(su, m, g, w.K);
      c.x[u][m] = bld16(xbuf, o == kPastEnd ? kPastEnd : row_off + o, 0);
    }
  }
}

template <int WT, int U>
__device__ __forceinline__ void stream_compute(const StreamChunk<WT, U>& c, int s, int s1, f32x4& acc) {
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (s + u < s1) {  // uniform
      if constexpr (WT == W_BF16) {
        acc = mfma16(c.x[u][0], as_bf16x8(c.w[u]), acc);
      } else {
        const float sc = scale_of_word(c.sc[u], s + u);
#pragma unroll
        for (int m = 0; m < 4; ++m) acc = mfma16(c.x[u][m], fp4x8_to_bf16x8(c.w[u][m], sc), acc);
      }
    }
  }
}

// acc += tokens . (row tile)^T over the steps [s0, s1): two chunks alternate, the next
// one in flight while one is multiplied.
template <int WT>
__device__ __forceinline__ void stream_tile(const Mat& w, int tile, int s0, int s1, __amdgpu_buffer_rsrc_t xbuf,
                                            int row_off, f32x4& acc) {
  constexpr int U = WT == W_BF16 ? 8 : 4;
  if (s0 >= s1) return;
  StreamChunk<WT, U> c0, c1;
  stream_load(c0, w, tile, s0, s1, xbuf, row_off);
  for (int s = s0; s < s1; s += 2 * U) {
    if (s + U < s1) stream_load(c1, w, tile, s + U, s1, xbuf, row_off);
    stream_compute(c0, s, s1, acc);
    if (s + 2 * U < s1) stream_load(c0, w, tile, s + 2 * U, s1, xbuf, row_off);
    if (s + U < s1) stream_compute(c1, s + U, s1, acc);
  }
}

}  // namespace moe
