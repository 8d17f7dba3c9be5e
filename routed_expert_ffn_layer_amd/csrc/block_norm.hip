// block_norm.hip -- the boundary of two blocks in one pass over the rows:
//     n  = norm_post(block)                           none, RMS or layer norm
//     r' = res_scale * res + block_scale * gate * n   (gate: per channel or per token and channel)
//     x  = norm_pre(r')
//
// Memory bound: block, res and, if given, gate rows are read once, r' and x written once, and
// a row stays in registers between its two norms (the next block's norm is taken from the f32
// row, not from its rounding to the stored type).  One row belongs to one wave, or to one
// workgroup of up to 16 waves for wide rows and small batches; a lane holds up to 4 groups of 8
// consecutive elements.
//
// Statistics in f32.  RMS: sum of squares.  Layer norm: mean first, then the sums of d = v - mean
// and of d^2, three reductions in all; the mean of d is what rounding left in the first mean, and is taken
// from d afterwards, so large offsets cost no digits.  Sums that leave the f32 range (elements
// past 2^63, or with a tiny eps below 2^-45) are formed again with the row scaled by a power of
// two, a branch that the whole row takes or leaves.
#include "kernels.hpp"
#include "row_io.hpp"

namespace moe {

namespace {

constexpr int kBnMaxWaves = 16;

// `a` reduced over the threads of a row; every thread gets it.  `red`: a float for each wave of the workgroup, of
// this reduction alone.
template <bool WAVE_ROW, typename Op>
__device__ __forceinline__ float row_reduce(float a, Op op, float* red) {
  a = reduce64(a, op);
  if constexpr (!WAVE_ROW) {
    const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63, nw = blockDim.x >> 6;
    if (lane == 0) red[wv] = a;
    lds_barrier();
    a = reduce16((lane & 15) < nw ? red[lane & 15] : 0.0f, op);  // sums, and maxima of magnitudes: 0 changes neither
  }
  return a;
}

// Mean square (RMS) or variance (layer norm) of the row s * v, plus eps (of the scaled row); mean + rest is the mean
// that a layer norm takes off.
template <int NV, bool WAVE_ROW>
__device__ __forceinline__ float statistics(const float (&v)[NV][8], int kind, float s, float eps, int H, int col0,
                                            int step, float (*red)[kBnMaxWaves], float& mean, float& rest) {
  // d below and in normalize() have to take off the same rounded mean: no fusing of a * inv_h into v - mean
#pragma clang fp contract(off)
  const float inv_h = 1.0f / (float)H;
  float a = 0.0f, b = 0.0f;
  mean = rest = 0.0f;
  if (kind == kNormLayer) {
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) a = fmaf(v[c][i], s, a);  // 0 past the row's end
    mean = row_reduce<WAVE_ROW>(a, Add(), red[0]) * inv_h;
    a = b = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = col0 + c * step + i < H ? fmaf(v[c][i], s, -mean) : 0.0f;
        a += d;
        b = fmaf(d, d, b);
      }
    rest = row_reduce<WAVE_ROW>(a, Add(), red[1]) * inv_h;
    b = row_reduce<WAVE_ROW>(b, Add(), red[2]);
    const float var = fmaf(-rest, rest, b * inv_h);
    return (var < 0.0f ? 0.0f : var) + eps;  // a NaN stays one
  }
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = v[c][i] * s;
      b = fmaf(d, d, b);
    }
  return row_reduce<WAVE_ROW>(b, Add(), red[0]) * inv_h + eps;
}

// v <- norm(v) * w (+ b); elements past the row's end stay 0.
template <int NV, bool WAVE_ROW>
__device__ __forceinline__ void normalize(float (&v)[NV][8], int kind, const float* __restrict__ w,
                                          const float* __restrict__ b, float eps, int H, int col0, int step,
                                          float (*red)[kBnMaxWaves]) {
  float mean, rest;
  float q = statistics<NV, WAVE_ROW>(v, kind, 1.0f, eps, H, col0, step, red, mean, rest);
  if (!(q >= 0x1p-90f && q < 0x1p126f)) {  // out of range, infinite or NaN
    float m = sqrtf(eps);
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[c][i]));
    m = row_reduce<WAVE_ROW>(m, Max(), red[3]);
    if (m > 0.0f && m < INFINITY) {  // else the definition's own infinities and NaN
      int e;
      frexpf(m, &e);
      const float s = ldexpf(1.0f, min(-e, 126));
      const float root = sqrtf(eps) * s;  // at most 1, where s^2 alone may pass the f32 range
      // red[0] to red[2] again: the maximum's barrier came after their last reads
      q = statistics<NV, WAVE_ROW>(v, kind, s, root * root, H, col0, step, red, mean, rest);
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= s;
    }
  }
  const float inv = 1.0f / sqrtf(q);
  if (kind == kNormLayer) {
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = col0 + c * step + i < H ? (v[c][i] - mean - rest) * inv : 0.0f;
  } else {
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= inv;
  }
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int col = col0 + c * step, n = H - col;
    if (n <= 0) continue;
    float wv[8];
    if (w) {
      load8(w + col, n, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= wv[i];
    }
    if (b) {
      load8(b + col, n, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] += wv[i];
    }
  }
}

// NV: groups of 8 elements a thread holds.  WAVE_ROW: a row per wave (4 rows a workgroup),
// else a row per workgroup.
template <int NV, bool WAVE_ROW, typename BT, typename RT, typename XT>
__global__ __launch_bounds__(WAVE_ROW ? 256 : 1024) void block_norm_kernel(BlockNormArgs a) {
  __shared__ float red[2][4][kBnMaxWaves];
  const int per_row = WAVE_ROW ? 64 : blockDim.x;
  const int64_t t = WAVE_ROW ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (WAVE_ROW && t >= a.T) return;  // no barriers in this form
  const int H = a.H, col0 = (WAVE_ROW ? threadIdx.x & 63 : threadIdx.x) * 8, step = per_row * 8;
  float v[NV][8], r[NV][8];
  const BT* brow = static_cast<const BT*>(a.block) + t * a.b_ld;
  const RT* rrow = static_cast<const RT*>(a.res) + t * a.r_ld;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int col = col0 + c * step, n = H - col;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = r[c][i] = 0.0f;
    if (n <= 0) continue;
    if (a.block) load8(brow + col, n, v[c]);
    if (a.res) load8(rrow + col, n, r[c]);
  }
  if (a.block) {
    if (a.post_kind != kNormNone)
      normalize<NV, WAVE_ROW>(v, a.post_kind, a.post_w, a.post_b, a.eps, H, col0, step, red[0]);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = col0 + c * step, n = H - col;
      if (n <= 0) continue;
      float g[8];
      if (a.gate) {
        if (a.gate_bf16)
          load8(static_cast<const uint16_t*>(a.gate) + t * a.gate_ld + col, n, g);
        else
          load8(static_cast<const float*>(a.gate) + t * a.gate_ld + col, n, g);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = a.gate ? v[c][i] * g[i] : v[c][i];
        // without a residual nothing is added (0 * inf would be NaN)
        v[c][i] = a.res ? fmaf(a.block_scale, u, a.res_scale * r[c][i]) : a.block_scale * u;
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = a.res_scale * r[c][i];
  }
  // res_out and x may lie on the rows read above: a thread writes the columns it has read
  if (a.res_out) {
    RT* row = static_cast<RT*>(a.res_out) + t * a.ro_ld;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = col0 + c * step, n = H - col;
      if (n > 0) store8(row + col, n, v[c]);
    }
  }
  if (a.x) {
    if (a.pre_kind != kNormNone)
      normalize<NV, WAVE_ROW>(v, a.pre_kind, a.pre_w, a.pre_b, a.eps, H, col0, step, red[1]);
    XT* row = static_cast<XT*>(a.x) + t * a.x_ld;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = col0 + c * step, n = H - col;
      if (n > 0) store8(row + col, n, v[c]);
    }
  }
}

template <typename BT, typename RT, typename XT>
hipError_t launch_typed(const BlockNormArgs& a, hipStream_t st) {
  const int groups = (a.H + 7) / 8;
  if (groups <= 64) {
    hipLaunchKernelGGL((block_norm_kernel<1, true, BT, RT, XT>), dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, st, a);
  } else if (groups <= 1024) {
    const int threads = (groups + 63) / 64 * 64;
    hipLaunchKernelGGL((block_norm_kernel<1, false, BT, RT, XT>), dim3((unsigned)a.T), dim3(threads), 0, st, a);
  } else if (groups <= 2048) {
    const int threads = (groups + 127) / 128 * 64;
    hipLaunchKernelGGL((block_norm_kernel<2, false, BT, RT, XT>), dim3((unsigned)a.T), dim3(threads), 0, st, a);
  } else {
    const int threads = (groups + 255) / 256 * 64;
    hipLaunchKernelGGL((block_norm_kernel<4, false, BT, RT, XT>), dim3((unsigned)a.T), dim3(threads), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, bool block_bf16, bool res_bf16, bool x_bf16, hipStream_t st) {
  typedef uint16_t B;
  typedef float F;
  switch ((block_bf16 ? 4 : 0) + (res_bf16 ? 2 : 0) + (x_bf16 ? 1 : 0)) {
    case 0: return launch_typed<F, F, F>(a, st);
    case 1: return launch_typed<F, F, B>(a, st);
    case 2: return launch_typed<F, B, F>(a, st);
    case 3: return launch_typed<F, B, B>(a, st);
    case 4: return launch_typed<B, F, F>(a, st);
    case 5: return launch_typed<B, F, B>(a, st);
    case 6: return launch_typed<B, B, F>(a, st);
    default: return launch_typed<B, B, B>(a, st);
  }
}

}  // namespace moe
