// linear.hip -- y = act(x W^T + bias) + res for f32 or bf16 weights stored as they come, one row of W
// after another.
//
// Two kernels.  linear_stream_kernel: every wave multiplies 16 RT weight rows by 16 TT tokens over its
// part of K with operands straight from memory in the matrix instructions' order, and the waves of a
// workgroup, which split K between them, add up in LDS.  There is no barrier before that sum and no
// staging, so the weights stream at the rate of memory: for few tokens, where the weights are the work,
// and for f32, whose matrix instructions are slow enough (1/16 of bf16's rate) to be fed this way at any
// size.  linear_tile_kernel: for many tokens in bf16, where the matrix instructions are the work:
// workgroup tiles staged through LDS.
//
// A 64-byte piece of a row is one step of the stream kernel: lane group g = lane / 16 holds bytes
// 16 g .. 16 g + 15 of it (8 bf16 or 4 f32) for row lane % 16, of weights and tokens alike.  In bf16
// that is the operand of one v_mfma_f32_16x16x32_bf16, in f32 of four v_mfma_f32_16x16x4_f32 (the
// k-th of them takes element k of the four lane groups).  Sums in f32, in an order fixed by the shape.
#include "ffn_common.hpp"
#include "kernels.hpp"
#include "row_io.hpp"

namespace moe {

namespace {

// 0.5 erfc(|z|) for z = v / sqrt(2): Abramowitz and Stegun 7.1.26, erf within 1.5e-7.
__device__ __forceinline__ float half_erfc(float z) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, z, 1.0f));
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  return 0.5f * p * t * __builtin_amdgcn_exp2f(-z * z * 1.4426950408889634f);
}

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {  // one value for the whole launch
    case kActRelu: return v < 0.0f ? 0.0f : v;
    case kActSilu: return silu_f32(v);
    case kActGelu: {
      const float q = half_erfc(fabsf(v) * 0.70710678118654752f);  // probability beyond |v|
      return v * (v < 0.0f ? q : 1.0f - q);
    }
    case kActGeluTanh: {  // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
      const float u = 0.79788456080286536f * fmaf(0.044715f * v * v, v, v);
      return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -2.8853900817779268f));
    }
    default: return v;
  }
}

// Finished value of one element.
__device__ __forceinline__ void finish(const LinearArgs& a, int64_t t, int n, float v) {
  if (a.bias) v += a.bias[n];
  v = activate(v, a.act);
  if (a.res) {
    const int64_t at = t * a.r_ld + n;
    v += a.res_bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(a.res)[at]) : static_cast<const float*>(a.res)[at];
  }
  if (a.y_bf16)
    static_cast<uint16_t*>(a.y)[t * a.y_ld + n] = f32_to_bf16_rne(v);
  else
    static_cast<float*>(a.y)[t * a.y_ld + n] = v;
}

constexpr int kPast = 0x7ffffff0;  // an offset past the end of every buffer made here (under 2^30 bytes): reads as 0

template <bool BF16>
__device__ __forceinline__ f32x4 mma_step(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
}

// Tokens are the A operand, weight rows the B operand: lane l of the 16 x 16 result holds tokens
// 4 (l / 16) + v and weight row l % 16.
// RT, TT: 16-row tiles of W and of tokens a wave holds; U: steps whose operands load together; MAXW: waves
// at most.
template <bool BF16, int RT, int TT, int U, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void linear_stream_kernel(LinearArgs a, int n_tiles) {
  extern __shared__ float lds[];  // [waves][RT][TT][64][4]
  constexpr int ES = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const int n0 = (int)(blockIdx.x % n_tiles) * 16 * RT;
  const int64_t t0 = (int64_t)(blockIdx.x / n_tiles) * 16 * TT;
  const int row = lane & 15, g = lane >> 4;
  const int kbytes = a.K * ES;
  // the tile's rows, and nothing behind them
  const auto wbuf = make_rsrc(static_cast<const uint8_t*>(a.w) + n0 * a.w_ld * ES,
                              (min(a.N - n0, 16 * RT) - 1) * a.w_ld * ES + kbytes);
  const auto xbuf = make_rsrc(static_cast<const uint8_t*>(a.x) + t0 * a.x_ld * ES,
                              (min(a.T - (int)t0, 16 * TT) - 1) * a.x_ld * ES + kbytes);
  int woff[RT], xoff[TT];  // this lane's rows; rows past the end read as 0
#pragma unroll
  for (int i = 0; i < RT; ++i) woff[i] = n0 + 16 * i + row < a.N ? (int)((16 * i + row) * a.w_ld * ES) + 16 * g : kPast;
#pragma unroll
  for (int i = 0; i < TT; ++i) xoff[i] = t0 + 16 * i + row < a.T ? (int)((16 * i + row) * a.x_ld * ES) + 16 * g : kPast;
  const int steps = (kbytes + 63) / 64, rounds = (steps + U - 1) / U;
  f32x4 acc[RT][TT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 wf[2][U][RT], xf[2][U][TT];
  auto load = [&](int r, u32x4 (&w)[U][RT], u32x4 (&x)[U][TT]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = (r * U + u) * 64;
      const bool in = at + 16 * g < kbytes;  // whole 16-byte fragments: K is a multiple of one
#pragma unroll
      for (int i = 0; i < RT; ++i) w[u][i] = bld16(wbuf, in && woff[i] != kPast ? woff[i] + at : kPast, 0);
#pragma unroll
      for (int i = 0; i < TT; ++i) x[u][i] = bld16(xbuf, in && xoff[i] != kPast ? xoff[i] + at : kPast, 0);
    }
  };
  auto multiply = [&](const u32x4 (&w)[U][RT], const u32x4 (&x)[U][TT]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = mma_step<BF16>(x[u][j], w[u][i], acc[i][j]);
  };
  int r = wv;
  if (r < rounds) load(r, wf[0], xf[0]);
  while (r < rounds) {
    if (r + nw < rounds) load(r + nw, wf[1], xf[1]);
    multiply(wf[0], xf[0]);
    r += nw;
    if (r >= rounds) break;
    if (r + nw < rounds) load(r + nw, wf[0], xf[0]);
    multiply(wf[1], xf[1]);
    r += nw;
  }
  f32x4* part = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) part[((wv * RT + i) * TT + j) * 64 + lane] = acc[i][j];
  lds_barrier();
  // element q of the tile: result (i, j), lane and register in order
  for (int q = threadIdx.x; q < RT * TT * 256; q += blockDim.x) {
    float s = 0.0f;
    for (int w = 0; w < nw; ++w) s += lds[w * RT * TT * 256 + q];
    const int v = q & 3, l = (q >> 2) & 63, ij = q >> 8;
    const int n = n0 + 16 * (ij / TT) + (l & 15);
    const int64_t t = t0 + 16 * (ij % TT) + 4 * (l >> 4) + v;
    if (n < a.N && t < a.T) finish(a, t, n, s);
  }
}

template <bool BF16, int RT, int TT, int U, int MAXW>
hipError_t launch_stream(const LinearArgs& a, hipStream_t st) {
  const int steps = (a.K * (BF16 ? 2 : 4) + 63) / 64;
  int waves = 1;  // no more than there are rounds of U steps
  while (waves < MAXW && waves * U < steps) waves *= 2;
  const int n_tiles = (a.N + 16 * RT - 1) / (16 * RT), t_tiles = (a.T + 16 * TT - 1) / (16 * TT);
  const int lds = waves * RT * TT * 1024;
  hipLaunchKernelGGL((linear_stream_kernel<BF16, RT, TT, U, MAXW>), dim3((unsigned)(n_tiles * t_tiles)), dim3(64 * waves), lds, st,
                     a, n_tiles);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_by_size(const LinearArgs& a, hipStream_t st) {
  if (a.T <= 16) return launch_stream<BF16, 1, 1, 8, 16>(a, st);
  if (a.T <= 32) return launch_stream<BF16, 2, 2, 4, 8>(a, st);
  return launch_stream<BF16, 4, 4, 2, 4>(a, st);
}

}  // namespace

hipError_t launch_linear(bool bf16, const LinearArgs& a, hipStream_t st) {
  return bf16 ? launch_by_size<true>(a, st) : launch_by_size<false>(a, st);
}

}  // namespace moe
