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
#include <stdlib.h>

#include <type_traits>

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

// The same for elements n .. n + 7 of token t, as far as they are in the row.
__device__ __forceinline__ void finish8(const LinearArgs& a, int64_t t, int n, float (&v)[8]) {
  const int left = a.N - n;
  if (a.bias) {
    float b[8];
    load8(a.bias + n, left, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = activate(v[i], a.act);
  if (a.res) {
    float r[8];
    if (a.res_bf16)
      load8(static_cast<const uint16_t*>(a.res) + t * a.r_ld + n, left, r);
    else
      load8(static_cast<const float*>(a.res) + t * a.r_ld + n, left, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  if (a.y_bf16)
    store8(static_cast<uint16_t*>(a.y) + t * a.y_ld + n, left, v);
  else
    store8(static_cast<float*>(a.y) + t * a.y_ld + n, left, v);
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

// ---------------------------------------------------------------------------
// Many tokens, bf16.  A workgroup of WN x WT waves computes BN weight rows by BT tokens; K goes in stages
// of 64, both operands' rows of a stage (128 bytes each) straight from memory into one of two LDS
// buffers, the next stage's loads in flight while this one is multiplied.  Matrix instruction
// v_mfma_f32_32x32x16_bf16, weights as A and tokens as B: a lane then holds 4 consecutive outputs of one
// token at a time, a vector store each.  Lane l supplies row l % 32, 16-byte piece 2 m + l / 32 of the row
// in k-step m.  Piece p of row r sits at position p ^ swz(r): the rows that one 128-bit LDS read touches
// land in distinct banks whether it is served 8 or 16 lanes at a time.
constexpr int kStage = 64;                // columns of a stage
constexpr int kStageBytes = kStage * 2;   // of one row

constexpr int kOutLd = 68;                // f32 of a row of results in LDS: 64 and 4 against bank conflicts
constexpr int kOutBytes = 32 * kOutLd * 4;

typedef __attribute__((address_space(3))) void* lds_ptr;

// A barrier and nothing more: waits are the caller's, memory accesses stay on their side.
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ int swz(int r) { return (r + (r >> 3)) & 7; }

template <int BN, int BT, int WN, int WT>
__global__ __launch_bounds__(64 * WN * WT) void linear_tile_kernel(LinearArgs a, int n_tiles, int t_tiles) {
  constexpr int W = WN * WT, RN = BN / WN / 32, RT = BT / WT / 32;  // 32-row tiles of a wave
  constexpr int ROWS = BN + BT, BUF = ROWS * kStageBytes, PIECES = ROWS / 8 / W;
  static_assert(BN % (8 * W) == 0 && BT % (8 * W) == 0, "a round of pieces is of one operand");
  static_assert(RN * RT >= RN + RT, "a product for each operand");
  extern __shared__ uint8_t smem[];
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6);
  const int rho = lane & 31, h = lane >> 5;
  // Workgroup b runs on XCD b % 8: each XCD takes a run of tiles, ordered so that neighbours share
  // rows in its L2: 4 weight tiles by all token tiles.
  int tn, tt;
  {
    const int total = n_tiles * t_tiles, x = blockIdx.x % 8, per = total / 8, more = total % 8;
    const int tile = x * per + min(x, more) + blockIdx.x / 8;
    const int group = tile / (4 * t_tiles), in = tile - group * 4 * t_tiles, wide = min(4, n_tiles - 4 * group);
    tn = 4 * group + in % wide;
    tt = in / wide;
  }
  const int n0 = tn * BN, t0 = tt * BT;
  const int wrows = min(BN, a.N - n0), xrows = min(BT, a.T - t0);
  const auto wbuf = make_rsrc(static_cast<const uint16_t*>(a.w) + n0 * a.w_ld, ((wrows - 1) * a.w_ld + a.K) * 2);
  const auto xbuf = make_rsrc(static_cast<const uint16_t*>(a.x) + t0 * a.x_ld, ((xrows - 1) * a.x_ld + a.K) * 2);
  // 1 KB pieces of 8 rows, wave wv takes pieces wv + W i; rows past the end repeat the last one, and in a
  // last, partial stage (of `tail` bytes) pieces past the end repeat the row's first one of the stage
  const int stages = (a.K + kStage - 1) / kStage, tail = (a.K % kStage) * 2;
  int voff[PIECES], past[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int row = 8 * (wv + W * i) + lane / 8, col = ((lane & 7) ^ swz(row)) * 16;
    voff[i] = (row < BN ? (int)(min(row, wrows - 1) * a.w_ld * 2) : (int)(min(row - BN, xrows - 1) * a.x_ld * 2)) + col;
    past[i] = tail && col >= tail ? col : 0;
  }
  // piece i of stage s; no branch: stages past the last repeat it
  auto load = [&](int s, uint8_t* buf, int i) {
    const int at = min(s, stages - 1), last = at == stages - 1 ? -1 : 0;
    const int piece = wv + W * i, from = voff[i] - (past[i] & last);
    if (W * i < BN / 8)  // known when the loops are unrolled
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wbuf, (lds_ptr)(buf + piece * 1024), 16, from, at * kStageBytes, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (lds_ptr)(buf + piece * 1024), 16, from, at * kStageBytes, 0, 0);
  };
  f32x16 acc[RN][RT];
#pragma unroll
  for (int i = 0; i < RN; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  // this lane's rows; swz(r + 32) = swz(r) ^ 4, and so the k-step's piece 2 m + h moves to m ^ 2
  const int wrow = (wv / WT) * (BN / WN) + rho, xrow = BN + (wv % WT) * (BT / WT) + rho;
  int wat[4], xat[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    wat[m] = wrow * kStageBytes + (((2 * m + h) ^ swz(wrow)) << 4);
    xat[m] = xrow * kStageBytes + (((2 * m + h) ^ swz(xrow)) << 4);
  }
  // operand q of step m: weight and token tiles by turns, in the order in which the products take them
  auto read = [&](const uint8_t* buf, int m, int q, bf16x8 (&A)[RN], bf16x8 (&B)[RT]) {
    if (q < RN)
      A[q] = as_bf16x8(*reinterpret_cast<const u32x4*>(buf + wat[m ^ (2 * (q & 1))] + q * 32 * kStageBytes));
    else
      B[q - RN] = as_bf16x8(*reinterpret_cast<const u32x4*>(buf + xat[m ^ (2 * ((q - RN) & 1))] + (q - RN) * 32 * kStageBytes));
  };
  // One step: the products of A and B; behind each of the first ones an operand of the next step (m of buffer
  // `next`) is read, and with LOAD pieces of stage s go out, so that neither keeps the matrix unit waiting.
  auto step = [&](auto LOAD, const uint8_t* next, int m, int s, uint8_t* into, const bf16x8 (&A)[RN], const bf16x8 (&B)[RT],
                  bf16x8 (&An)[RN], bf16x8 (&Bn)[RT]) {
#pragma unroll
    for (int p = 0; p < RN * RT; ++p) {
      const int i = p % RN, j = p / RN;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(A[i], B[j], acc[i][j], 0, 0, 0);
      if (p < RN + RT) read(next, m, p, An, Bn);
      if constexpr (decltype(LOAD)::value) {
#pragma unroll
        for (int d = p * PIECES / (RN * RT); d < (p + 1) * PIECES / (RN * RT); ++d) load(s, into, d);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Steps m = 0 .. 3 of stage s.  The first step's operands are read behind the barrier that ends the stage
  // before, under that stage's last products.  The barrier also frees the stage's buffer, for the loads of
  // stage s + 2.
#pragma unroll
  for (int i = 0; i < PIECES; ++i) load(0, smem, i);
#pragma unroll
  for (int i = 0; i < PIECES; ++i) load(1, smem + BUF, i);
  const int whole = tail ? stages - 1 : stages;
  bf16x8 A[2][RN], B[2][RT];
  constexpr int kOneStage = 0x0f70 | (PIECES & 15) | PIECES >> 4 << 14;  // vmcnt(PIECES)
  __builtin_amdgcn_s_waitcnt(kOneStage);  // stage 0 has landed, stage 1 is on its way
  block_barrier();
#pragma unroll
  for (int q = 0; q < RN + RT; ++q) read(smem, 0, q, A[0], B[0]);
  const std::true_type with_loads;
  const std::false_type without;
  for (int s = 0; s < whole; ++s) {
    uint8_t *buf = smem + (s & 1) * BUF, *other = smem + ((s + 1) & 1) * BUF;
    step(without, buf, 1, 0, buf, A[0], B[0], A[1], B[1]);
    step(without, buf, 2, 0, buf, A[1], B[1], A[0], B[0]);
    step(without, buf, 3, 0, buf, A[0], B[0], A[1], B[1]);
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0): own loads of stage s + 1, own reads of stage s
    block_barrier();
    step(with_loads, other, 0, s + 2, buf, A[1], B[1], A[0], B[0]);  // past the last stage: read and not used
  }
  if (tail) {
    const uint8_t* buf = smem + ((stages - 1) & 1) * BUF;  // landed and visible since the last barrier
    for (int m = 0; 32 * m < tail; ++m) {
      const int p = 2 * m + h;  // computed here: m is no constant
#pragma unroll
      for (int i = 0; i < RN; ++i) {
        const int r = wrow + 32 * i;
        const u32x4 v = *reinterpret_cast<const u32x4*>(buf + r * kStageBytes + ((p ^ swz(r)) << 4));
        A[0][i] = as_bf16x8(p * 16 < tail ? v : u32x4{0, 0, 0, 0});
      }
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int r = xrow + 32 * j;
        const u32x4 v = *reinterpret_cast<const u32x4*>(buf + r * kStageBytes + ((p ^ swz(r)) << 4));
        B[0][j] = as_bf16x8(p * 16 < tail ? v : u32x4{0, 0, 0, 0});
      }
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int i = 0; i < RN; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(A[0][i], B[0][j], acc[i][j], 0, 0, 0);
    }
  }
  // Results: 32 tokens by 64 weight rows at a time through the wave's own part of LDS, so that a lane
  // finishes 8 consecutive outputs and the rows of res and y are read and written in whole lines.
  static_assert(W * kOutBytes <= 2 * BUF && RN % 2 == 0, "the results' part of LDS");
  __builtin_amdgcn_s_waitcnt(0x0f70);  // the loads past the last stage have landed
  __syncthreads();                     // and nobody reads a stage any more
  float* out = reinterpret_cast<float*>(smem + wv * kOutBytes);
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int i2 = 0; i2 < RN; i2 += 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& c = acc[i2 + i][j];  // lane: token rho, rows 8 q + 4 h + 0 .. 3
          *reinterpret_cast<f32x4*>(out + rho * kOutLd + 32 * i + 8 * q + 4 * h) =
              f32x4{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
        }
      __builtin_amdgcn_wave_barrier();
      const int n = n0 + (wv / WT) * (BN / WN) + 32 * i2 + 8 * (lane & 7);
      for (int u = lane >> 3; u < 32; u += 8) {
        const int t = t0 + (wv % WT) * (BT / WT) + 32 * j + u;
        if (t >= a.T || n >= a.N) continue;
        float v[8];
        const f32x4 lo = *reinterpret_cast<const f32x4*>(out + u * kOutLd + 8 * (lane & 7));
        const f32x4 hi = *reinterpret_cast<const f32x4*>(out + u * kOutLd + 8 * (lane & 7) + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = lo[e];
          v[4 + e] = hi[e];
        }
        finish8(a, t, n, v);
      }
      __builtin_amdgcn_wave_barrier();
    }
}

template <int BN, int BT, int WN, int WT>
hipError_t launch_tile(const LinearArgs& a, hipStream_t st) {
  const int n_tiles = (a.N + BN - 1) / BN, t_tiles = (a.T + BT - 1) / BT;
  constexpr int lds = 2 * (BN + BT) * kStageBytes;
  hipLaunchKernelGGL((linear_tile_kernel<BN, BT, WN, WT>), dim3((unsigned)(n_tiles * t_tiles)), dim3(64 * WN * WT), lds, st, a,
                     n_tiles, t_tiles);
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
  if (bf16 && a.T > 128) {
    const char* e = getenv("LIN");
    const int v = e ? atoi(e) : 0;
    if (v == 1) return launch_tile<256, 256, 2, 2>(a, st);
    if (v == 2) return launch_tile<128, 128, 2, 2>(a, st);
    if (v == 3) return launch_tile<256, 128, 2, 2>(a, st);
    if (v == 4) return launch_tile<256, 256, 4, 2>(a, st);
    if (v == 5) return launch_tile<128, 128, 2, 1>(a, st);
    if (v == 6) return launch_by_size<true>(a, st);
    return launch_tile<256, 256, 2, 4>(a, st);
  }
  return bf16 ? launch_by_size<true>(a, st) : launch_by_size<false>(a, st);
}

}  // namespace moe
