// linear.hip -- y = act(x W^T + bias) + res for f32 or bf16 weights stored as they come, one row of W
// after another.
//
// Three kernels.  linear_stream_kernel, for up to 8 tokens: every wave multiplies 16 weight rows by 4 or 8 tokens over its
// part of K, operands straight from memory in registers, and the waves of a workgroup, which split K between
// them, add up in LDS.  linear_small_kernel, for up to 16 tokens or small results: the same with 16 tokens and operands
// through LDS, each wave for itself.  linear_tile_kernel, for all else: tiles staged through LDS by the whole workgroup,
// from 32 x 32 (weights are the work: many small workgroups, deep in flight) to 256 x 256 (the matrix instructions
// are).  Sums in f32, in an order fixed by the shape.
//
// Measured on an MI355X, bf16, x weights x K (plain library product beside it): 1 x 4096 x 4096 4.5 us (10.5),
// 16 x 512 x 4096 4.9 (8.0), 16 x 12288 x 4096 17.5 (21), 64 x 4096 x 4096 9.1 (19), 4 x 65536 x 4096 87 (124; 537 MB
// at 6.2 TB/s), 256 x 4096 x 4096 16.3 (19.7), 1024 x 4096 x 4096 35.6 (37.4), 4096 x 8192 x 4096 220 (177 once both
// are warm; 1.25 PFLOP/s), 512 x 256 x 4096 9.4 (8.3); f32: 4 x 512 x 4096 7.4 (9.9), 16 x 64 x 4096 7.9 (9.7), 32 x 2048 x 2048 6.0 (8.9),
// 64 x 4096 x 4096 25 (22), 4096 x 4096 x 4096 944 (920; 146 TFLOP/s).
//
// Against the library's product of the same type over 42 pairs of weights (100 to 12288) and K (512 to 16384), as the
// geometric mean of the times' ratios, both captured and warm: bf16 0.67 to 0.80 for 1 to 256 tokens, 0.99 for 512, 1.04 and 1.06
// for 1024 and 2048, 1.11 and 1.16 for 4096 and 8192; f32 0.78 to 0.93 for 1 to 256, 1.10 to 1.18 from 512 on.  Farthest behind:
// large results of short K, whose prologue and epilogue no product covers (bf16 8192 x 12288 x 512 187 us and 114, 1024 x 12288 x
// 1024 48 and 30), and few results of deep K, where the library spreads K over the chip and adds up in memory (bf16
// 512 x 100 x 8192 14 and 8.6, f32 1024 x 100 x 16384 84 and 43, 85 x 864 x 14400 56 and 41, 256 x 12288 x 4096 254 and 180).
#include "ffn_common.hpp"
#include "kernels.hpp"
#include "row_io.hpp"

#include <type_traits>

namespace moe {

namespace {

// P(Z > a) of a normal Z, a >= 0: t P(t) e^(-a^2 / 2) with t = 1 / (1 + 0.375 a / sqrt(2)).  P, of degree 8, is fitted to
// erfc(z) e^(z^2) / 2 over z = a / sqrt(2) in [0, 9.5] for the least relative error, 1.2e-8, so that the tail keeps its
// digits: within (1.5 a^2 + 24) 2^-24 relative, of which the exponent's roundings are the first term.  (4096 x 8192 x 4096 with GELU
// 239 us; 237 with degree 4 and 1.5e-7 absolutely, which at -8 is 1e-2 of the value.)
__device__ __forceinline__ float normal_tail(float a) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.26516504294495533f, a, 1.0f));
  float p = fmaf(3.084828891e-02f, t, -1.440376043e-01f);
  p = fmaf(p, t, 2.169467062e-01f);
  p = fmaf(p, t, -1.155380011e-01f);
  p = fmaf(p, t, 1.374219209e-01f);
  p = fmaf(p, t, 6.051953882e-02f);
  p = fmaf(p, t, 1.027151942e-01f);
  p = fmaf(p, t, 1.053167507e-01f);
  p = fmaf(p, t, 1.058072075e-01f);
  return p * t * __builtin_amdgcn_exp2f(a * a * -0.72134752044448170f);
}

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {  // one value for the whole launch
    case kActRelu: return v < 0.0f ? 0.0f : v;
    case kActSilu: return silu_f32(v);
    case kActGelu: {
      const float q = normal_tail(fabsf(v));
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

// Elements n .. n + 7 of token t of res as memory holds them, so that they can be on their way while others are
// worked on; 0 where there are none.
struct Residual8 {
  Raw8<uint16_t> b;
  Raw8<float> f;
  __device__ __forceinline__ void load(const LinearArgs& a, int64_t t, int n, bool live) {
    const int left = live && a.res ? a.N - n : 0;
    const int64_t at = left > 0 ? t * a.r_ld + n : 0;
    if (a.res_bf16)
      b.load<false>(static_cast<const uint16_t*>(a.res) + at, left);
    else
      f.load<false>(static_cast<const float*>(a.res) + at, left);
  }
  __device__ __forceinline__ float value(const LinearArgs& a, int i) const { return a.res_bf16 ? b[i] : f[i]; }
};

// Finished values of elements n .. n + 7 of token t from sums v, bias b and residual r.
__device__ __forceinline__ void finish8(const LinearArgs& a, int64_t t, int n, float (&v)[8], const float (&b)[8],
                                        const Residual8& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += b[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = activate(v[i], a.act);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += r.value(a, i);
  if (a.y_bf16)
    store8(static_cast<uint16_t*>(a.y) + t * a.y_ld + n, a.N - n, v);
  else
    store8(static_cast<float*>(a.y) + t * a.y_ld + n, a.N - n, v);
}

constexpr int kPast = 0x7ffffff0;  // an offset past the end of every buffer made here (under 2^30 bytes): reads as 0

// ---------------------------------------------------------------------------
// Up to 4 or 8 tokens, 16 weight rows a workgroup; its waves take steps of 256 bytes of K in turn, the next step's loads
// on their way while one is multiplied, and add up in LDS.
//
// Memory is quick where four neighbouring lanes read 64 bytes in a row (with neighbours in different rows a CU
// got 35 GB/s, 1 x 4096 x 4096 took 7.4 us; now 4.5).  So load i of a step gives lane (g, b, c), g = lane / 16,
// b = lane / 4 % 4, c = lane % 4, the 16-byte piece 4 g + c of weight row 4 b + i, or of token X b + i of X = TOKENS / 4
// loads.  v_mfma_f32_16x16x32_bf16 (f32: four v_mfma_f32_16x16x4_f32) takes lane % 16 for its row, so "row" (b, c) of a
// product is piece c of row b alone: of its 16 x 16 results those with the same c on both sides count, four of
// which make up a sum, and every weight load is multiplied with every token load.  That is X times the products of
// a layout by rows, with no work between load and product (moving the registers into that layout takes 64 moves and
// choices for 4 KB: 4 x 4096 x 4096 6.5 us instead of 4.8).
//
// 8 waves, or as many as there are steps (weights from memory: 1 x 4096 x 4096 8.1 us, in 16 waves 9.1, in 4 9.0).
// ---------------------------------------------------------------------------
// v of another lane of the quad.
template <int CTRL>
__device__ __forceinline__ unsigned quad_u32(unsigned v) {
  return (unsigned)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
__device__ __forceinline__ unsigned from_xor1(unsigned v) { return quad_u32<0xb1>(v); }
__device__ __forceinline__ unsigned from_xor2(unsigned v) { return quad_u32<0x4e>(v); }

// c += A . B: 16 rows by 16 over four pieces, 32 bf16 or 16 f32.
template <bool BF16>
__device__ __forceinline__ f32x4 mma_pieces(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
}

constexpr int kStreamWaves = 8;

template <bool BF16, int TOKENS>
__global__ __launch_bounds__(64 * kStreamWaves) void linear_stream_kernel(LinearArgs a) {
  __shared__ float part[kStreamWaves][TOKENS * 16];
  constexpr int ES = BF16 ? 2 : 4, X = TOKENS / 4;
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const int g = lane >> 4, b = lane >> 2 & 3, c = lane & 3;
  const int n0 = (int)blockIdx.x * 16;
  const int kbytes = a.K * ES;
  // the tile's rows, and nothing behind them
  const auto wbuf = make_rsrc(static_cast<const uint8_t*>(a.w) + n0 * a.w_ld * ES,
                              (min(a.N - n0, 16) - 1) * a.w_ld * ES + kbytes);
  const auto xbuf = make_rsrc(a.x, (a.T - 1) * a.x_ld * ES + kbytes);
  // this lane's pieces of the first step; rows past the end read as 0
  const int piece = 16 * (4 * g + c);
  unsigned wo[4], xo[X];
#pragma unroll
  for (int i = 0; i < 4; ++i) wo[i] = n0 + 4 * b + i < a.N ? (int)((4 * b + i) * a.w_ld * ES) + piece : kPast;
#pragma unroll
  for (int i = 0; i < X; ++i) xo[i] = X * b + i < a.T ? (int)((X * b + i) * a.x_ld * ES) + piece : kPast;
  f32x4 acc[X][4];
#pragma unroll
  for (auto& row : acc)
#pragma unroll
    for (f32x4& v : row) v = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 wf[2][4], xf[2][X];
  auto load = [&](int s, u32x4 (&w)[4], u32x4 (&x)[X]) {
    const int at = s * 256;  // kPast + at stays past the end
    const bool in = at + piece < kbytes;  // whole pieces: K is a multiple of one
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = bld16(wbuf, (int)((in ? wo[i] : kPast) + at), 0);
      if (i < X) x[i] = bld16(xbuf, (int)((in ? xo[i] : kPast) + at), 0);
    }
  };
  auto multiply = [&](const u32x4 (&w)[4], const u32x4 (&x)[X]) {
#pragma unroll
    for (int j = 0; j < X; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = mma_pieces<BF16>(x[j], w[i], acc[j][i]);
  };
  const int steps = (kbytes + 255) / 256;
  int s = wv;
  if (s < steps) load(s, wf[0], xf[0]);
  while (s < steps) {
    if (s + nw < steps) load(s + nw, wf[1], xf[1]);
    multiply(wf[0], xf[0]);
    s += nw;
    if (s >= steps) break;
    if (s + nw < steps) load(s + nw, wf[0], xf[0]);
    multiply(wf[1], xf[1]);
    s += nw;
  }
  // The wave's sums, [token][row].  Lane l of a product holds its rows (tokens) 4 g + v, column (weight row) l % 16.
#pragma unroll
  for (int j = 0; j < X; ++j) {
    f32x4 sum;  // token (g, j), rows (b, i)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4& v = acc[j][i];
      const float lo = c & 1 ? v[1] : v[0], hi = c & 1 ? v[3] : v[2];
      float mine = c & 2 ? hi : lo;  // row c of column c
      mine += __uint_as_float(from_xor1(__float_as_uint(mine)));
      mine += __uint_as_float(from_xor2(__float_as_uint(mine)));
      sum[i] = mine;
    }
    if (c == 0) *reinterpret_cast<f32x4*>(&part[wv][(X * g + j) * 16 + 4 * b]) = sum;
  }
  lds_barrier();
  for (int q = threadIdx.x; q < TOKENS * 16; q += blockDim.x) {
    float sum = 0.0f;
    for (int w = 0; w < nw; ++w) sum += part[w][q];
    const int n = n0 + q % 16, t = q / 16;
    if (n < a.N && t < a.T) finish(a, t, n, sum);
  }
}

template <bool BF16, int TOKENS>
hipError_t launch_stream(const LinearArgs& a, hipStream_t st) {
  const int steps = (a.K * (BF16 ? 2 : 4) + 255) / 256;
  int waves = 1;
  while (waves < kStreamWaves && waves < steps) waves *= 2;
  hipLaunchKernelGGL((linear_stream_kernel<BF16, TOKENS>), dim3((unsigned)((a.N + 15) / 16)), dim3(64 * waves), 0, st, a);
  return hipGetLastError();
}

constexpr int kRow = 128;  // bytes of a row in a stage

typedef __attribute__((address_space(3))) void* lds_ptr;

// A barrier and nothing more: waits are the caller's, memory accesses stay on their side.
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// s_waitcnt with at most N vector loads outstanding; LGKM: and no LDS access.
template <int N, bool LGKM>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  constexpr int imm = (N & 15) | (N >> 4) << 14 | (LGKM ? 0x0070 : 0x0f70);
  __builtin_amdgcn_s_waitcnt(imm);
}

// A 128-bit LDS read is served 16 lanes at a time, over 256 bytes of banks: lanes 0-3, 12-15 and 20-27
// of each half first, then the others.  The XOR term gives the rows of each of these groups places of their own
// (no bank conflicts counted; (r + r / 8) % 8 for 128-byte rows cost 4 cycles a read).
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// ---------------------------------------------------------------------------
// More tokens with few results: 16 weight rows by 16 tokens a workgroup.  Each of its 8 waves works alone, on steps of
// 128 bytes of K in turn: both operands' rows straight from memory into its own two LDS buffers, 8 rows of whole lines a
// load, one step ahead; no barrier until the waves add up.  Operands as in the tile kernel below, places by the same swz:
// lane l reads piece 4 m + l / 16 of row l % 16 for product m.  Of a step's time the loads take 64 cycles of its CU and
// the f32 products as many.  Measured (operands in registers instead, moved into place; plain library product): f32
// 16 x 64 x 4096 7.9 us (11.5; 9.7), 32 x 2048 x 2048 6.0 (8.4; 8.9), bf16 16 x 2048 x 4096 5.5 (6.2; 8.2).  Three or four
// buffers instead of two: one workgroup in a CU, 16 x 65536 x 4096 102 us becomes 118 and 120.
// ---------------------------------------------------------------------------
constexpr int kSmallBuf = 32 * kRow;

template <bool BF16>
__global__ __launch_bounds__(64 * kStreamWaves) void linear_small_kernel(LinearArgs a, int n_tiles) {
  extern __shared__ uint8_t smem[];
  constexpr int ES = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const int n0 = (int)(blockIdx.x % n_tiles) * 16, t0 = (int)(blockIdx.x / n_tiles) * 16;
  const int kbytes = a.K * ES, wrows = min(16, a.N - n0), xrows = min(16, a.T - t0);
  const auto wbuf = make_rsrc(static_cast<const uint8_t*>(a.w) + n0 * a.w_ld * ES, (wrows - 1) * a.w_ld * ES + kbytes);
  const auto xbuf = make_rsrc(static_cast<const uint8_t*>(a.x) + t0 * a.x_ld * ES, (xrows - 1) * a.x_ld * ES + kbytes);
  uint8_t* mine = smem + wv * 2 * kSmallBuf;
  // load i of a step: rows 8 i .. 8 i + 7 of weights, then of tokens; rows past the end repeat the last one
  const int col0 = ((lane & 7) ^ swz(lane >> 3)) * 16, col1 = ((lane & 7) ^ swz(8 + (lane >> 3))) * 16;
  unsigned off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 8 * (i & 1) + (lane >> 3);
    off[i] = (unsigned)((i < 2 ? min(row, wrows - 1) * a.w_ld : min(row, xrows - 1) * a.x_ld) * ES) + (i & 1 ? col1 : col0);
  }
  auto load = [&](int s, uint8_t* buf) {  // steps past the last read nothing
    const int at = s * kRow;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int from = (int)(at + (i & 1 ? col1 : col0) < kbytes ? off[i] + at : kPast);
      if (i < 2)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(wbuf, (lds_ptr)(buf + i * 1024), 16, from, 0, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (lds_ptr)(buf + i * 1024), 16, from, 0, 0, 0);
    }
  };
  const int row = lane & 15, g = lane >> 4;
  int place[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) place[m] = row * kRow + (((4 * m + g) ^ swz(row)) << 4);
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  const int steps = (kbytes + kRow - 1) / kRow;
  load(wv, mine);
  for (int s = wv, slot = 0; s < steps; s += nw, slot ^= 1) {
    load(s + nw, mine + (slot ^ 1) * kSmallBuf);
    wait_loads<4, false>();  // this step has landed
    asm volatile("" ::: "memory");
    const uint8_t* buf = mine + slot * kSmallBuf;
    u32x4 w[2], x[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      w[m] = *reinterpret_cast<const u32x4*>(buf + place[m]);
      x[m] = *reinterpret_cast<const u32x4*>(buf + 16 * kRow + place[m]);
    }
    if (s == steps - 1) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (s * kRow + 16 * (4 * m + g) >= kbytes) w[m] = x[m] = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) acc[m] = mma_pieces<BF16>(x[m], w[m], acc[m]);
    asm volatile("" ::: "memory");
    wait_loads<63, true>();  // the buffer is read: the next load may go into it
    asm volatile("" ::: "memory");
  }
  wait_loads<0, true>();  // no load is on its way to the sums' place
  asm volatile("" ::: "memory");
  float* part = reinterpret_cast<float*>(mine);
#pragma unroll
  for (int v = 0; v < 4; ++v) part[(4 * g + v) * 16 + row] = acc[0][v] + acc[1][v];
  lds_barrier();
  for (int q = threadIdx.x; q < 256; q += blockDim.x) {
    float sum = 0.0f;
    for (int w = 0; w < nw; ++w) sum += reinterpret_cast<const float*>(smem + w * 2 * kSmallBuf)[q];
    const int n = n0 + q % 16, t = t0 + q / 16;
    if (n < a.N && t < a.T) finish(a, t, n, sum);
  }
}

template <bool BF16>
hipError_t launch_small(const LinearArgs& a, hipStream_t st) {
  const int steps = (a.K * (BF16 ? 2 : 4) + kRow - 1) / kRow;
  int waves = 1;
  while (waves < kStreamWaves && waves < steps) waves *= 2;
  const int n_tiles = (a.N + 15) / 16, t_tiles = (a.T + 15) / 16;
  hipLaunchKernelGGL(linear_small_kernel<BF16>, dim3((unsigned)(n_tiles * t_tiles)), dim3(64 * waves),
                     waves * 2 * kSmallBuf, st, a, n_tiles);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// More tokens.  A workgroup computes BN weight rows by BT tokens on WN x WT x WK waves: WN x WT of them side by
// side, and WK that share a part of the tile and split K between them (their sums meet in LDS at the end).  K
// goes in stages of 128 bytes, both operands' rows of a stage straight from memory into one of D LDS buffers,
// the next ones in flight while one is multiplied.  Matrix instruction v_mfma_f32_32x32x16_bf16 or
// v_mfma_f32_32x32x2_f32, weights as A and tokens as B.  Lane l supplies row l % 32, 16-byte piece 2 m + l / 32 of
// the row in step m of the stage.  Piece p of row r sits at place p ^ swz(r).
//
// Each step is laid out by hand: a product, an operand read of the next step, a load of a later stage, the next
// product, .. (reads, loads and products one after the other: 4096 x 8192 x 4096 in 267 us, so 220).  What bounds
// the largest tile now is the loads: with the same products and none of them in the loop it takes 193 us, with all
// of them from the same stage 216; without the barrier nothing changes.  The matrix unit is busy in 68 to 72% of
// the cycles (the library's 87%), at a clock of 1.7 to 1.8 GHz (counter runs).  Measured and not kept: 4 waves of 128 x 128 (324 us:
// one wave per SIMD), stages of 64 bytes with 4 or 5 buffers (231), workgroups starting at other columns (neutral
// or slower).
// ---------------------------------------------------------------------------
// Results of a wave in LDS: 32 tokens by one or two 32-row tiles, padded against bank conflicts.
constexpr int out_ld(int tiles) { return 32 * (tiles % 2 ? 1 : 2) + 4; }
constexpr int out_bytes(int tiles) { return 32 * out_ld(tiles) * 4; }

// acc += A . B over 32 bytes of K: 16 bf16, or 8 f32 in four products (the k-th of both halves' pieces each).
template <bool BF16>
__device__ __forceinline__ f32x16 mma_tile(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
}

template <bool BF16, int BN, int BT, int WN, int WT, int WK, int D>
__global__ __launch_bounds__(64 * WN * WT * WK) void linear_tile_kernel(LinearArgs a, int n_tiles, int t_tiles) {
  constexpr int W = WN * WT * WK, RN = BN / WN / 32, RT = BT / WT / 32;  // 32-row tiles of a wave
  constexpr int ES = BF16 ? 2 : 4, PPR = kRow / 16, RPP = 64 / PPR;      // 16-byte pieces of a row; rows of 1 KB
  constexpr int BUF = (BN + BT) * kRow, LOADS = (BN + BT) / RPP / W;      // a stage's loads of a wave, 1 KB each
  constexpr int S = kRow / 32 / WK, P = RN * RT;                           // steps of a wave in a stage, products in a step
  static_assert(BN % (RPP * W) == 0 && BT % (RPP * W) == 0, "a round of loads is of one operand");
  extern __shared__ uint8_t smem[];
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6);
  const int rho = lane & 31, h = lane >> 5;
  const int wk = wv % WK, wt = wv / WK % WT, wn = wv / WK / WT;
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
  const int64_t w_step = a.w_ld * ES, x_step = a.x_ld * ES;
  const int kbytes = a.K * ES;
  const auto wbuf = make_rsrc(static_cast<const uint8_t*>(a.w) + n0 * w_step, (wrows - 1) * w_step + kbytes);
  const auto xbuf = make_rsrc(static_cast<const uint8_t*>(a.x) + t0 * x_step, (xrows - 1) * x_step + kbytes);
  // Load i of wave wv fills rows RPP (wv + W i) .. of the stage's buffer; rows past the end repeat the last
  // one, and in a last, partial stage (of `tail` bytes) pieces past the end repeat the row's first one of the stage.
  const int stages = (kbytes + kRow - 1) / kRow, tail = kbytes % kRow;
  int voff[LOADS], past[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int row = RPP * (wv + W * i) + lane / PPR, col = ((lane % PPR) ^ swz(row)) * 16;
    voff[i] = (row < BN ? (int)(min(row, wrows - 1) * w_step) : (int)(min(row - BN, xrows - 1) * x_step)) + col;
    past[i] = tail && col >= tail ? col : 0;
  }
  // load i of stage s; no branch: stages past the last repeat it
  auto load = [&](int s, uint8_t* buf, int i) {
    const int at = min(s, stages - 1), last = at == stages - 1 ? -1 : 0;
    const int from = voff[i] - (past[i] & last);
    if (W * i < BN / RPP)  // known when the loops are unrolled
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wbuf, (lds_ptr)(buf + (wv + W * i) * 1024), 16, from, at * kRow, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (lds_ptr)(buf + (wv + W * i) * 1024), 16, from, at * kRow, 0, 0);
  };
  f32x16 acc[RN][RT];
#pragma unroll
  for (int i = 0; i < RN; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  // this lane's rows (swz is the same 32 rows on) in the wave's steps wk, wk + WK, ..
  const int wrow = wn * (BN / WN) + rho, xrow = BN + wt * (BT / WT) + rho;
  int wat[S], xat[S];
#pragma unroll
  for (int m = 0; m < S; ++m) {
    const int p = 2 * (wk + WK * m) + h;
    wat[m] = wrow * kRow + ((p ^ swz(wrow)) << 4);
    xat[m] = xrow * kRow + ((p ^ swz(xrow)) << 4);
  }
  // operand q of the wave's step m: weight tiles, then token tiles
  auto read = [&](const uint8_t* buf, int m, int q, u32x4 (&A)[RN], u32x4 (&B)[RT]) {
    if (q < RN)
      A[q] = *reinterpret_cast<const u32x4*>(buf + wat[m] + q * 32 * kRow);
    else
      B[q - RN] = *reinterpret_cast<const u32x4*>(buf + xat[m] + (q - RN) * 32 * kRow);
  };
  // The loads of a stage go out in parts, under the steps that follow the barrier that frees their buffer, so that
  // their issue keeps up with the products: over S steps, with two buffers over two, which leaves the last part
  // two steps to land in.
  constexpr int SPREAD = D > 2 ? S : 2;
  // One step: the products of A and B; behind each of them operands of the next step (m of buffer `next`) are
  // read and part e of stage s's loads goes out, into `into`, so that neither keeps the matrix unit waiting.  Part
  // 0 belongs to a stage's last step: after its first X products the next stage has to have landed, and this
  // one's buffer is free.
  auto step = [&](const uint8_t* next, int m, auto E, int s, uint8_t* into, const u32x4 (&A)[RN], const u32x4 (&B)[RT],
                  u32x4 (&An)[RN], u32x4 (&Bn)[RT]) {
    constexpr int e = decltype(E)::value;
    constexpr int X = e == 0 ? (P > 4 ? 4 : 0) : 0, per = (RN + RT + P - X - 1) / (P - X);  // operands a product
    constexpr int lo = e < SPREAD ? e * LOADS / SPREAD : 0, hi = e < SPREAD ? (e + 1) * LOADS / SPREAD : 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int i = p % RN, j = p / RN;
      if (e == 0 && p == X) {
        wait_loads<(D - 2) * LOADS, true>();  // own loads of the next stage, own reads of this one
        block_barrier();
      }
      acc[i][j] = mma_tile<BF16>(A[i], B[j], acc[i][j]);
#pragma unroll
      for (int q = (p - X) * per; q < (p - X + 1) * per; ++q)
        if (q >= 0 && q < RN + RT) read(next, m, q, An, Bn);
#pragma unroll
      for (int d = lo + max(p - X, 0) * (hi - lo) / (P - X); d < lo + max(p - X + 1, 0) * (hi - lo) / (P - X); ++d)
        load(s, into, d);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
#pragma unroll
    for (int i = 0; i < (d < D - 1 ? LOADS : LOADS / SPREAD); ++i) load(d, smem + d * BUF, i);
  const int whole = tail ? stages - 1 : stages;
  u32x4 A[2][RN], B[2][RT];
  wait_loads<(D - 2) * LOADS + LOADS / SPREAD, false>();  // stage 0 has landed
  block_barrier();
#pragma unroll
  for (int q = 0; q < RN + RT; ++q) read(smem, 0, q, A[0], B[0]);
  // The first step's operands are read behind the barrier that ends the stage before, under that stage's
  // last products.
  uint8_t *buf = smem, *freed = smem + (D - 1) * BUF;
  auto stage = [&](int s, auto FIRST) {  // FIRST: the operand set that holds the stage's first step
    constexpr int f = decltype(FIRST)::value;
    uint8_t* other = buf == smem + (D - 1) * BUF ? smem : buf + BUF;
    auto early = [&](auto E) {  // step E - 1 of the stage
      constexpr int e = decltype(E)::value;
      if constexpr (e < S)
        step(buf, e, E, s + D - 1, freed, A[(e - 1 + f) & 1], B[(e - 1 + f) & 1], A[(e + f) & 1], B[(e + f) & 1]);
    };
    early(std::integral_constant<int, 1>());
    early(std::integral_constant<int, 2>());
    early(std::integral_constant<int, 3>());
    step(other, 0, std::integral_constant<int, 0>(), s + D, buf, A[(S - 1 + f) & 1], B[(S - 1 + f) & 1], A[(S + f) & 1],
         B[(S + f) & 1]);
    freed = buf;
    buf = other;  // past the last stage its operands are read and not used
  };
  static_assert(S <= 4, "steps of a stage");
  const std::integral_constant<int, 0> even;
  const std::integral_constant<int, S & 1> odd;
  int s = 0;
  for (; s + 1 < whole; s += 2) {
    stage(s, even);
    stage(s + 1, odd);
  }
  if (s < whole) stage(s, even);
  if (tail) {  // landed and visible since the last barrier
    for (int m = wk; 32 * m < tail; m += WK) {
      const int p = 2 * m + h;
#pragma unroll
      for (int q = 0; q < RN + RT; ++q) {
        const int r = q < RN ? wrow + 32 * q : xrow + 32 * (q - RN);
        u32x4 v = *reinterpret_cast<const u32x4*>(buf + r * kRow + ((p ^ swz(r)) << 4));
        if (p * 16 >= tail) v = u32x4{0, 0, 0, 0};
        if (q < RN)
          A[0][q] = v;
        else
          B[0][q - RN] = v;
      }
#pragma unroll
      for (int p2 = 0; p2 < P; ++p2)
        acc[p2 % RN][p2 / RN] = mma_tile<BF16>(A[0][p2 % RN], B[0][p2 / RN], acc[p2 % RN][p2 / RN]);
    }
  }
  // Results: 32 tokens by up to 64 weight rows at a time through LDS, so that a lane finishes 8
  // consecutive outputs and the rows of res and y are read and written in whole lines.  The WK waves of a part
  // share its tokens out between them.  The residual of a slice is on its way while the slice before it
  // is finished (4096 x 8192 x 4096 with activation and residual: 243 us; fetched for its own slice 250, for each of a
  // wave's passes 260).
  constexpr int SL = RN % 2 ? 1 : 2, LD = out_ld(RN), LANES = 4 * SL;  // tiles of a slice; lanes a token
  constexpr int PER = 64 / LANES, PASSES = PER * WK >= 32 ? 1 : 32 / (PER * WK), SLICES = RN / SL * RT;
  constexpr int kOutBytes = out_bytes(RN);
  const int u0 = wk * PER + lane / LANES;
  auto first_row = [&](int q) { return n0 + wn * (BN / WN) + 32 * SL * (q / RT) + 8 * (lane % LANES); };
  auto first_token = [&](int q) { return t0 + wt * (BT / WT) + 32 * (q % RT) + u0; };
  Residual8 r[2][PASSES];
  auto fetch = [&](int q) {
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
      const int t = first_token(q) + u * PER * WK, n = first_row(q);
      r[q & 1][u].load(a, t, n, u0 < 32 && t < a.T && n < a.N);
    }
  };
  fetch(0);
  wait_loads<0, false>();  // the loads past the last stage have landed
  __syncthreads();         // and nobody reads a stage any more
  float* out = reinterpret_cast<float*>(smem + wv * kOutBytes);
  const float* part = reinterpret_cast<const float*>(smem + (wv - wk) * kOutBytes);
  float bias[8] = {};
#pragma unroll
  for (int q = 0; q < SLICES; ++q) {
    const int i2 = q / RT * SL, j = q % RT, n = first_row(q);
    if (j == 0 && a.bias && n < a.N) load8(a.bias + n, a.N - n, bias);
#pragma unroll
    for (int i = 0; i < SL; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const f32x16& c = acc[i2 + i][j];  // lane: token rho, rows 8 v + 4 h + 0 .. 3
        *reinterpret_cast<f32x4*>(out + rho * LD + 32 * i + 8 * v + 4 * h) =
            f32x4{c[4 * v], c[4 * v + 1], c[4 * v + 2], c[4 * v + 3]};
      }
    if (q + 1 < SLICES) fetch(q + 1);
    if constexpr (WK > 1)
      lds_barrier();
    else
      __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < PASSES; ++u) {
      const int t = first_token(q) + u * PER * WK;
      if (u0 >= 32 || t >= a.T || n >= a.N) continue;
      float v[8] = {};
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        const float* p = part + k * (kOutBytes / 4) + (u0 + u * PER * WK) * LD + 8 * (lane % LANES);
        const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] += lo[e];
          v[4 + e] += hi[e];
        }
      }
      finish8(a, t, n, v, bias, r[q & 1][u]);
    }
    if constexpr (WK > 1)
      lds_barrier();
    else
      __builtin_amdgcn_wave_barrier();
  }
}

template <bool BF16, int BN, int BT, int WN, int WT, int WK, int D>
hipError_t launch_tile(const LinearArgs& a, hipStream_t st) {
  const int n_tiles = (a.N + BN - 1) / BN, t_tiles = (a.T + BT - 1) / BT;
  constexpr int ring = D * (BN + BT) * kRow, out = WN * WT * WK * out_bytes(BN / WN / 32);
  constexpr int lds = ring > out ? ring : out;
  hipLaunchKernelGGL((linear_tile_kernel<BF16, BN, BT, WN, WT, WK, D>), dim3((unsigned)(n_tiles * t_tiles)),
                     dim3(64 * WN * WT * WK), lds, st, a, n_tiles, t_tiles);
  return hipGetLastError();
}

// Tile shapes, by the time that a stage (128 bytes of K) of a round of 256 workgroups, one for each CU, takes: us,
// measured at K = 4096 with 256 workgroups (the first four, by the matrix unit; the others, by the latency of a
// stage).  The shape whose rounds come out cheapest is taken.  Over T = 16 .. 4096 and N = 500 .. 20000 it is within 8% of the
// best of the seven at bf16 and K = 4096; at K = 1024, where a round is mostly prologue and epilogue, that it does not
// count, within 13% (1000 x 12288: 46.6 us, 41.2 in tiles of 256 x 256); f32 at K = 2048 within 23% (700 x 4096: 143 us, 116
// in tiles of 64 x 32, of which a CU holds several, which it does not count either).  Single shapes lose up to 8 times.
struct LinearForm {
  int rows, tokens;
  float us[2];  // f32, bf16; of the tile shapes
  hipError_t (*launch[2])(const LinearArgs&, hipStream_t);
};
#define TILE(BN, BT, F, B, ...) \
  {BN, BT, {F, B}, {launch_tile<false, BN, BT, __VA_ARGS__>, launch_tile<true, BN, BT, __VA_ARGS__>}}
const LinearForm kShapes[] = {
    TILE(256, 256, 7.4f, 1.77f, 4, 2, 1, 2), TILE(256, 128, 3.8f, 0.99f, 4, 2, 1, 3),
    TILE(128, 128, 2.0f, 0.55f, 2, 2, 2, 4), TILE(128, 64, 1.1f, 0.37f, 2, 1, 2, 4),
    TILE(64, 64, 0.57f, 0.25f, 1, 1, 4, 4),  TILE(64, 32, 0.31f, 0.18f, 1, 1, 4, 5),
    TILE(32, 32, 0.20f, 0.14f, 1, 1, 4, 8),
};
#undef TILE
const LinearForm kStream4 = {16, 4, {}, {launch_stream<false, 4>, launch_stream<true, 4>}};
const LinearForm kStream8 = {16, 8, {}, {nullptr, launch_stream<true, 8>}};
const LinearForm kSmall = {16, 16, {}, {launch_small<false>, launch_small<true>}};

// Up to 8 tokens (f32: 4) the stream kernel.  The small kernel takes up to 16, where the tiles' 32 token rows would be
// half of the loads (weights from memory, bf16: 16 x 4096 x 4096 9.7 us, 12 in tiles, 16 x 65536 x 4096 102 and 104; f32:
// 16 x 4096 x 4096 17.5 and 24), and few 16 x 16 tiles: a 32 x 32 tile there waits for one CU's loads or matrix unit
// while others have nothing to do.  bf16, up to one tile a CU: 64 x 512 x 4096 4.9 us, 8.7 in tiles of 32; up to two
// where K is short (100 x 600 x 2048 5.3 and 6.3, x 4096 7.4 and 8.8, but 1000 x 100 x 4096 12.3 and 9.0, 64 x 2048 x 16384
// 29 and 24).  f32, up to two: 64 x 64 x 14400 22 and 75, 256 x 512 x 4096 15.4 and 24.6; four: 64 x 4096 x 4096 41
// and 25.
const LinearForm& choose_form(bool bf16, int T, int N, int K) {
  const bool few = (int64_t)((N + 15) / 16) * ((T + 15) / 16) <= (bf16 && K > 2048 ? 256 : 512);
  if (T <= 4) return kStream4;
  if (bf16 && T <= 8) return kStream8;
  if (few || T <= 16) return kSmall;
  const LinearForm* best = nullptr;
  float least = 0.0f;
  for (const LinearForm& s : kShapes) {
    const int64_t tiles = (int64_t)((N + s.rows - 1) / s.rows) * ((T + s.tokens - 1) / s.tokens);
    const float us = (float)((tiles + 255) / 256) * s.us[bf16];
    if (!best || us < least) {
      best = &s;
      least = us;
    }
  }
  return *best;
}

}  // namespace

int linear_tile(bool bf16, int T, int N, int K) {
  const LinearForm& f = choose_form(bf16, T, N, K);
  return f.rows << 16 | f.tokens;
}

hipError_t launch_linear(bool bf16, const LinearArgs& a, hipStream_t st) {
  return choose_form(bf16, a.T, a.N, a.K).launch[bf16](a, st);
}

}  // namespace moe
