// w4.hip -- products with 4-bit weights for a few tokens: y = x . W^T (+ bias).
//
//   MXFP4: W[n][k] = E2M1(code) * 2^(scale[n][k/32] - 127)
//   INT4:  W[n][k] = s[n][k/G] * (q - z[n][k/G]),  q in 0..15
//
// Laid-out weights: tiles of 16 rows x 128 columns of 1 KB (row-tile major, then column
// step), so that a wave reads a tile as one contiguous KB and lane l's 16 bytes are the
// operands of four 32-column MFMAs.  MXFP4 keeps the layout of the expert slots.  An
// INT4 tile's fragment f = 16 g + row holds, in word m, the 8 codes of columns
// 32 m + 8 g .. + 7, so one MFMA covers 32 consecutive columns, one group or a part of
// one, and the group's scale is applied to its f32 sum: the operand stays the exact
// integer code, never a rounded product.  Inside a word, nibble 2 j is column j and nibble
// 2 j + 1 column 4 + j, so the bytes of (word & 0x0f0f0f0f) are columns 0 .. 3 and those of
// the shifted word columns 4 .. 7.
// Scale and zero of a group are one 32-bit word (two f16), four consecutive groups of
// a row side by side: per row tile, blocks of 4 groups x 16 rows, 256 bytes each.
//
// INT4 codes become bf16 through E4M3: a byte 0 .. 15 is q * 2^-9 in that format (the
// subnormals and the first binade are one linear run), so the scaled convert by 2^9
// gives q exactly, two per instruction.
//   sum_k x W = sum over groups s * (sum_k x q - z sum_k x)
// and sum_k x over the same 32 columns is one more MFMA with an all-ones operand.  That identity
// holds while nothing overflows: an infinite x makes both sums infinite and their difference NaN,
// and finite ones may pass the f32 range before the scale brings them back.  Either leaves the
// output infinite or NaN, so an output that is gets formed again from W itself (int4_redo).
//
// Times here and below: captured calls over enough weight sets to come from HBM, K = 4096.  Up to 16
// tokens the codes bound the product (MXFP4, 65536 rows, 16 tokens: 35.5 us, 83% of a large copy's rate);
// small matrices are bound by one launch and one round trip to memory (2048 x 2048: 3.7 us). 64 tokens over
// many rows are bound by the instructions that unpack, scale and multiply (INT4 in groups of 128, 65536 rows:
// 58 us, floor 32), and 17 to 64 over 2048 to 36000 rows by w4_wide's walk of the whole K in one wave: 64 tokens
// take 24 us at 4096 rows and 26 at 12288 (floors 2 and 6).
#include <type_traits>

#include "kernels.hpp"
#include "stream_tile.hpp"

namespace moe {

// More than 16 tokens: w4_few reads the codes once per 16 tokens, w4_wide once per 64 with blocks
// of 4 row tiles (4 waves of one) or 16 (8 waves of two, which read a token from LDS half as
// often).  Measured at K = 4096, us, for INT4 in groups of 128 / 64 / 32 and MXFP4:
//   64 tokens, N = 2048:   w4_few 15 / 15 / 16, 15     w4_wide 24 / 27 / 38, 19
//              N = 4096:          27 / 27 / 30, 27             24 / 27 / 38, 20
//   24 tokens, N = 6000:          16 / 16 / 18, 16             15 / 17 / 20, 13
//              N = 12288:         19 / 20 / 22, 18             16 / 18 / 21, 14
// Above 32 tokens a CU holds two blocks of 4 row tiles, so 2048 tiles are one round of them; up to 32 it
// holds more, by the registers (groups of 32 one: there the second limit costs 20 us at N = 36000).
//   64 tokens, N = 24576:  4 tiles 39 / 56 / 60, 30     16 tiles 48 / 51 / 65, 36
//              N = 36000:          59 / 83 / 90, 48              49 / 52 / 67, 38
//              N = 65536:          82 / 122 / 117, 62            60 / 65 / 75, 47
//   32 tokens, N = 36000:          32 / 41 / 62, 30              33 / 34 / 42, 29
//              N = 65536:          47 / 56 / 84, 41              43 / 44 / 48, 39
constexpr int kW4WideWork = 1024;    // row tiles x passes of 16 tokens from which w4_wide is taken
constexpr int kW4WideTiles = 2049;   // row tiles from which its blocks have 16
constexpr int kW4WideTiles32 = 2800; // the same up to 32 tokens

static size_t w4_code_bytes(int N, int K) { return (size_t)((N + 15) / 16) * ((K + 127) / 128) * 1024; }

static size_t w4_scale_bytes(int fmt, int N, int K, int group) {
  const size_t rt = (N + 15) / 16;
  if (fmt == W_MXFP4) return rt * (((K + 127) / 128 + 15) / 16) * 1024;
  const size_t groups = (K + group - 1) / group;
  return rt * ((groups + 3) / 4) * 256;
}

size_t w4_bytes(int fmt, int N, int K, int group) { return w4_code_bytes(N, K) + w4_scale_bytes(fmt, N, K, group); }

// ---------------------------------------------------------------------------
// Layout.  A thread lays out a 16-byte code fragment at a time, then 16 bytes (MXFP4) or one word
// of scales, and goes on by the size of the grid: a launch holds fewer than 2^32 threads, a
// large matrix more fragments.  Rows past N and columns past K become zero codes and zero scales.
// ---------------------------------------------------------------------------
constexpr unsigned kPackBlocks = 1 << 16;  // 256 MiB of codes a turn
static dim3 pack_grid(size_t threads) {
  const size_t blocks = (threads + 255) / 256;
  return dim3((unsigned)(blocks < kPackBlocks ? blocks : kPackBlocks));
}

// The 8 codes of 4 source bytes (element 2i in the low nibble of byte i) in the word order
// above: nibble 2j holds element j, nibble 2j + 1 element 4 + j (j < 4).
__device__ __forceinline__ uint32_t int4_word(uint32_t v) {
  uint32_t o = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) o |= ((v >> (4 * j)) & 15u) << (8 * j) | ((v >> (16 + 4 * j)) & 15u) << (8 * j + 4);
  return o;
}

template <int FMT>
__global__ __launch_bounds__(256) void w4_pack_codes(const uint8_t* __restrict__ codes, int N, int K, uint8_t* w) {
  const int nk = (K + 127) / 128;
  const int64_t total = (int64_t)((N + 15) / 16) * nk * 64;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int f = i & 63, r = f & 15, g = f >> 4;
    const int64_t ts = i >> 6;
    const int step = ts % nk;
    const int64_t row = ts / nk * 16 + r;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (row < N) {
      const uint8_t* src = codes + row * (K / 2);
      if constexpr (FMT == W_MXFP4) {
        if (step * 128 + 32 * g < K) v = ldg16(src + step * 64 + 16 * g);
      } else {
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (step * 128 + 32 * m < K)
            v[m] = int4_word(*reinterpret_cast<const uint32_t*>(src + step * 64 + 16 * m + 4 * g));
      }
    }
    *reinterpret_cast<u32x4*>(w + i * 16) = v;
  }
}

__global__ __launch_bounds__(256) void w4_pack_mx_scales(const uint8_t* __restrict__ scales, int N, int K, uint8_t* w) {
  const int nb = ((K + 127) / 128 + 15) / 16, groups = K / 32;
  const int64_t total = (int64_t)((N + 15) / 16) * nb * 64;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int f = i & 63, r = f & 15, g = f >> 4;
    const int blk = (i >> 6) % nb;
    const int64_t row = (i >> 6) / nb * 16 + r;
    for (int b = 0; b < 16; ++b) {
      const int grp = (blk * 16 + b) * 4 + g;
      w[i * 16 + b] = row < N && grp < groups ? scales[row * groups + grp] : 0;
    }
  }
}

__global__ __launch_bounds__(256) void w4_pack_int4_scales(const uint16_t* __restrict__ scales,
                                                           const uint8_t* __restrict__ zeros, int N, int groups,
                                                           uint8_t* w) {
  const int nb = (groups + 3) / 4;
  const int64_t total = (int64_t)((N + 15) / 16) * nb * 64;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int q = i & 3, r = (i >> 2) & 15;
    const int grp = (i >> 6) % nb * 4 + q;
    const int64_t row = (i >> 6) / nb * 16 + r;
    uint32_t word = 0;
    if (row < N && grp < groups) {
      const int z = zeros ? zeros[row * groups + grp] : 8;
      word = scales[row * groups + grp] | (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)z) << 16;
    }
    reinterpret_cast<uint32_t*>(w)[i] = word;
  }
}

hipError_t launch_w4_pack(int fmt, const uint8_t* codes, const void* scales, const uint8_t* zeros, int N, int K,
                          int group, uint8_t* w, hipStream_t st) {
  const size_t cb = w4_code_bytes(N, K), sb = w4_scale_bytes(fmt, N, K, group);
  const dim3 gc = pack_grid(cb / 16), block(256);
  if (fmt == W_MXFP4) {
    hipLaunchKernelGGL(w4_pack_codes<W_MXFP4>, gc, block, 0, st, codes, N, K, w);
    hipLaunchKernelGGL(w4_pack_mx_scales, pack_grid(sb / 16), block, 0, st, static_cast<const uint8_t*>(scales), N, K,
                       w + cb);
  } else {
    hipLaunchKernelGGL(w4_pack_codes<W_INT4>, gc, block, 0, st, codes, N, K, w);
    hipLaunchKernelGGL(w4_pack_int4_scales, pack_grid(sb / 4), block, 0, st, static_cast<const uint16_t*>(scales), zeros,
                       N, (K + group - 1) / group, w + cb);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Product.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bf16x8 int4x8_to_bf16x8(uint32_t w) {
  const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  u32x4 v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ float f16_lo(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)w); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16)); }


// Parameters of two consecutive column steps (the first one even): words of 32 bits per
// lane, this lane's weight row.  MXFP4: one word of E8M0 bytes.  INT4: 128 / G words a step.
template <int FMT, int G>
struct W4Params {
  static constexpr int words = FMT == W_MXFP4 ? 1 : 256 / G;
  uint32_t v[words];
};

// Byte offsets of a row tile's codes and parameters, per tile.
struct W4Shape {
  int nk, code_tile, par_tile;
  size_t par_at;
  __device__ __forceinline__ W4Shape(int fmt, int N, int K, int G) {
    nk = (K + 127) / 128;
    code_tile = nk * 1024;
    par_at = (size_t)((N + 15) / 16) * code_tile;
    par_tile = fmt == W_MXFP4 ? (nk + 15) / 16 * 1024 : ((K + G - 1) / G + 3) / 4 * 256;
  }
};

// Loads the parameters of steps `step`, `step` + 1 of a tile whose parameters are `buf`.
template <int FMT, int G>
__device__ __forceinline__ void load_params(W4Params<FMT, G>& p, __amdgpu_buffer_rsrc_t buf, int step, bool live) {
  const int lane = threadIdx.x & 63;
  if constexpr (FMT == W_MXFP4) {
    p.v[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(buf, lane * 16, live ? step / 16 * 1024 + step % 16 / 4 * 4 : 0, 0);
  } else {
    // word (group % 4) of block group / 4, 16 bytes a row
    const int vo = (lane & 15) * 16;
    if constexpr (G == 128) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                                                    buf, vo, live ? step / 4 * 256 + step % 4 * 4 : 0, 0));
      p.v[0] = v[0];
      p.v[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < W4Params<FMT, G>::words / 4; ++i) {
        const u32x4 v = bld16(buf, vo, live ? (step * (128 / G) / 4 + i) * 256 : 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) p.v[4 * i + j] = v[j];
      }
    }
  }
}

// acc[r][nt] += x . W^T over step u (0 or 1) of a pair of steps, for R row tiles (codes
// w[r], parameters p[r]) and NT token tiles; frag(nt, m) is the token fragment m of the
// step.  INT4: a group's products and activation sums are formed first (d, xs), then
// scale (d - zero xs) is added to the f32 accumulator.
template <int FMT, int G, int R, int NT, typename Frag>
__device__ __forceinline__ void w4_step(f32x4 (&acc)[R][NT], const u32x4 (&w)[R],
                                        const W4Params<FMT, G> (&p)[R], int u, int step, const Frag& frag) {
  if constexpr (FMT == W_MXFP4) {
    float sc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) sc[r] = scale_of_word(p[r].v[0], step);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      u32x4 x[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[nt] = frag(nt, m);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bf16x8 b = fp4x8_to_bf16x8(w[r][m], sc[r]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[r][nt] = mfma16(x[nt], b, acc[r][nt]);
      }
    }
  } else {
    constexpr int B = G / 32;  // products per group
    const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 d[R][NT], xs[NT];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      u32x4 x[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        x[nt] = frag(nt, m);
        xs[nt] = mfma16(x[nt], as_bf16x8(ones), m % B ? xs[nt] : zero);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bf16x8 b = int4x8_to_bf16x8(w[r][m]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) d[r][nt] = mfma16(x[nt], b, m % B ? d[r][nt] : zero);
      }
      if (m % B == B - 1) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint32_t pw = p[r].v[(4 * u + m) / B];
          const float sc = f16_lo(pw), z = f16_hi(pw);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[r][nt][v] = fmaf(sc, fmaf(-z, xs[nt][v], d[r][nt][v]), acc[r][nt][v]);
        }
      }
    }
  }
}

template <bool BF16OUT>
__device__ __forceinline__ void store_y(const W4Args& a, int64_t row, int64_t col, float y) {
  if (a.bias) y += a.bias[col];
  if (BF16OUT)
    static_cast<uint16_t*>(a.y)[row * a.y_ld + col] = f32_to_bf16_rne(y);
  else
    static_cast<float*>(a.y)[row * a.y_ld + col] = y;
}

// An INT4 output that came out infinite or NaN, again from the definition: s (q - z) is exact in
// f32 (f16 times an integer of 9 bits), its products with x are added in ascending k with one
// rounding each.  Runs when a wave's last output is written, with nothing else in registers, so that
// the ordinary path pays a comparison per output (within 1% at 1 to 64 tokens).  It is bound by a
// single lane's unpacking: a batch with one infinite token 785 us instead of 35 (65536 x 4096, 16 tokens),
// 270 instead of 60 (64 tokens); outputs that are NaN end with the first NaN.
template <int G, bool BF16OUT>
__device__ __forceinline__ void int4_redo(const W4Args& a, const W4Shape& sh, int64_t t, int64_t col) {
  if (BF16OUT) {
    if (isfinite(bf16_bits_to_f32(static_cast<const uint16_t*>(a.y)[t * a.y_ld + col]))) return;
  } else {
    if (isfinite(static_cast<const float*>(a.y)[t * a.y_ld + col])) return;
  }
  const int64_t tile = col >> 4;
  const int row = (int)(col & 15);
  const uint8_t* codes = a.w + (size_t)tile * sh.code_tile + row * 16;
  const uint8_t* par = a.w + sh.par_at + (size_t)tile * sh.par_tile + row * 16;
  const uint16_t* x = a.x + t * a.x_ld;
  float y = 0.f;
#pragma unroll 1
  for (int k0 = 0; k0 < a.K && y == y; k0 += 32) {  // NaN stays NaN
    const uint32_t pw = *reinterpret_cast<const uint32_t*>(par + k0 / G / 4 * 256 + k0 / G % 4 * 4);
    const float sc = f16_lo(pw), z = f16_hi(pw);
    u32x4 xv[4];
    uint32_t q[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      xv[g] = ldg16(x + k0 + 8 * g);
      q[g] = *reinterpret_cast<const uint32_t*>(codes + (size_t)(k0 / 128) * 1024 + g * 256 + k0 % 128 / 32 * 4);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // column j in nibble 2 j, column 4 + j in nibble 2 j + 1
        const float code = (float)(q[g] >> (8 * (j & 3) + (j & 4)) & 15u);
        const float xj = __uint_as_float(j & 1 ? xv[g][j / 2] & 0xffff0000u : xv[g][j / 2] << 16);
        y = fmaf(sc * (code - z), xj, y);
      }
  }
  store_y<BF16OUT>(a, t, col, y);
}

// Up to 16 tokens.  The waves of a block split K in pairs of column steps, so a wave's token
// fragments are the same for every row tile: it keeps them in registers (NC pairs of steps;
// NC = 0: K too long, they are read again for every tile) and streams the codes of the
// block's contiguous range of row tiles through a few buffers of two steps.  At the end
// of a tile the block adds the waves' parts in LDS, in ascending order (two buffers, one
// barrier per tile, which waits for no load).  Up to 4 VN tokens, in a quad of lanes the
// same token would be held 4 / VN times: there each lane loads another fragment (VN = 4:
// every lane its own token).
template <int VN, int NC>
struct W4Bufs {  // as many as the registers of 16 waves hold
  static constexpr int value = NC == 0 || (NC == 2 && VN == 4) ? 2 : VN == 4 ? 3 : 4;
};


// acc += x . W^T over one step of a row tile (codes w, parameters p), for up to 4 VN tokens
// whose fragments are quad-loaded: x[l] holds fragments l * NA + f, f < NA = 4 / VN, fragment
// f in the quads' lanes f VN .. f VN + VN - 1.  A product with fragment f's weights takes
// x[l] as it is and is right in its elements from f VN on; pick() gathers them.
template <int FMT, int G, int VN>
__device__ __forceinline__ void w4_step_few(float (&acc)[VN], f32x4 (&part)[4 / VN], u32x4 w, const W4Params<FMT, G>& p,
                                            int u, int step, const u32x4 (&x)[VN]) {
  constexpr int NA = 4 / VN;
  if constexpr (FMT == W_MXFP4) {
    const float sc = scale_of_word(p.v[0], step);
#pragma unroll
    for (int m = 0; m < 4; ++m) part[m % NA] = mfma16(x[m / NA], fp4x8_to_bf16x8(w[m], sc), part[m % NA]);
  } else {
    constexpr int B = G / 32;  // products per group
    const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 d[4], xs[VN];
#pragma unroll
    for (int l = 0; l < VN; ++l) xs[l] = mfma16(x[l], as_bf16x8(ones), zero);
#pragma unroll
    for (int m = 0; m < 4; ++m) d[m] = mfma16(x[m / NA], int4x8_to_bf16x8(w[m]), zero);
#pragma unroll
    for (int m0 = 0; m0 < 4; m0 += B) {
      const uint32_t pw = p.v[(4 * u + m0) / B];
      const float sc = f16_lo(pw), z = f16_hi(pw);
#pragma unroll
      for (int v = 0; v < VN; ++v) {
        float ds = 0.f, xsum = 0.f;
#pragma unroll
        for (int m = m0; m < m0 + B; ++m) {
          const float dm = d[m][v + VN * (m % NA)], xm = xs[m / NA][v + VN * (m % NA)];
          ds = m == m0 ? dm : ds + dm;
          xsum = m == m0 ? xm : xsum + xm;
        }
        acc[v] = fmaf(sc, fmaf(-z, xsum, ds), acc[v]);
      }
    }
  }
}

template <int FMT, int G, int VN, int NC, bool BF16OUT>
__global__ __launch_bounds__(1024) void w4_few(W4Args a, int nc) {
  constexpr int NX = NC ? NC : 1, B = W4Bufs<VN, NC>::value;
  extern __shared__ float red[];  // [buffer][element v][part][lane]
  const int lane = threadIdx.x & 63, g = lane >> 4, kp = uniform(threadIdx.x >> 6), waves = uniform(blockDim.x >> 6);
  const int t0 = blockIdx.y * 16, m = min(16, a.T - t0), j = lane & 3, q4 = (lane & 15) >> 2;
  const W4Shape sh(FMT, a.N, a.K, G);
  const int tiles = (a.N + 15) / 16;
  const int lo = (int)((int64_t)blockIdx.x * tiles / gridDim.x), hi = (int)((int64_t)(blockIdx.x + 1) * tiles / gridDim.x);
  const int step0 = kp * nc * 2;

  // Token fragments: load l of a step holds fragment f of token tok for this lane.
  const int tok = min(q4 + 4 * (VN == 1 ? 0 : VN == 2 ? (j & 1) : j), m - 1);
  const __amdgpu_buffer_rsrc_t xbuf = make_rsrc(a.x + (size_t)t0 * a.x_ld, ((size_t)(m - 1) * a.x_ld + a.K) * 2);
  const int x_row = tok * (int)a.x_ld * 2;
  auto load_x = [&](u32x4(&x)[VN], int step) {
#pragma unroll
    for (int l = 0; l < VN; ++l) {
      const int f = VN == 1 ? j : VN == 2 ? 2 * l + (j >> 1) : l;
      const int o = frag_offset<FMT>(step, f, g, a.K);
      x[l] = bld16(xbuf, o == kPastEnd ? kPastEnd : x_row + o, 0);
    }
  };
  u32x4 xr[NX][2][VN];
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u) load_x(xr[c][u], step0 + 2 * c + u);
  }

  struct Buf {
    u32x4 w[2];
    W4Params<FMT, G> p;
    u32x4 x[NC ? 1 : 2][VN];
  };
  Buf buf[B];
  int iq = lo, ic = 0;
  auto issue = [&](Buf& b) {
    const int step = step0 + 2 * ic;
    const uint8_t* codes = a.w + (size_t)iq * sh.code_tile;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool live = iq < hi && step + u < sh.nk;
      b.w[u] = bld16(make_rsrc(codes, live ? sh.code_tile : 0), lane * 16, live ? (step + u) * 1024 : 0);
    }
    const bool live = iq < hi && step < sh.nk;
    load_params<FMT, G>(b.p, make_rsrc(a.w + sh.par_at + (size_t)iq * sh.par_tile, live ? sh.par_tile : 0), step, live);
    if constexpr (NC == 0) {
#pragma unroll
      for (int u = 0; u < 2; ++u) load_x(b.x[u], step + u);
    }
    if (++ic == nc) {
      ic = 0;
      ++iq;
    }
  };
#pragma unroll
  for (int b = 0; b < B; ++b) issue(buf[b]);
  // MXFP4, and 16 tokens, add up in the products' accumulators, INT4 in acc
  constexpr int NA = 4 / VN;
  float acc[VN];
  f32x4 sums[NA];
  auto clear = [&]() {
#pragma unroll
    for (int v = 0; v < VN; ++v) acc[v] = 0.f;
#pragma unroll
    for (int f = 0; f < NA; ++f) sums[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  clear();
  int q = lo, half = 0;
  uint64_t again = 0;  // INT4: lanes with an output to be formed again
  const int red_tile = VN * waves * 64;
  auto compute = [&](const Buf& b, int c, const u32x4(&x0)[VN], const u32x4(&x1)[VN]) {
    const int step = step0 + 2 * c;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (step + u >= sh.nk) continue;
      const u32x4(&x)[VN] = u ? x1 : x0;
      if constexpr (VN == 4) {  // every lane its own token: the products of a group chain
        const u32x4 w[1] = {b.w[u]};
        const W4Params<FMT, G> p[1] = {b.p};
        f32x4 a1[1][1] = {{sums[0]}};
        w4_step<FMT, G, 1, 1>(a1, w, p, u, step + u, [&](int, int f) { return x[f]; });
        sums[0] = a1[0][0];
      } else {
        w4_step_few<FMT, G, VN>(acc, sums, b.w[u], b.p, u, step + u, x);
      }
    }
  };
  auto tile_end = [&]() {  // returns whether a tile is left
    float* part = red + half * red_tile;
#pragma unroll
    for (int v = 0; v < VN; ++v) {
      float d = acc[v];
      if constexpr (FMT == W_MXFP4 || VN == 4) {
        d = sums[0][v];
#pragma unroll
        for (int f = 1; f < NA; ++f) d += sums[f][v + VN * f];
      }
      part[(v * waves + kp) * 64 + lane] = d;
    }
    clear();
    lds_barrier();
    // element v by wave (q VN + v) % waves: lane = (token % 4, row)
    for (int v = 0; v < VN; ++v) {
      if ((q * VN + v) % waves != kp) continue;
      float y = 0.f;
      for (int w = 0; w < waves; ++w) y += part[(v * waves + w) * 64 + lane];
      const int64_t col = (int64_t)q * 16 + (lane & 15);
      const bool mine = g + 4 * v < m && col < a.N;
      if (mine) store_y<BF16OUT>(a, t0 + g + 4 * v, col, y);
      if constexpr (FMT == W_INT4) again |= __ballot(mine && !isfinite(y));
    }
    half ^= 1;
    return ++q < hi;
  };
  if constexpr (NC > 0) {
    // buffer b holds chunk b % NC of its tile
    static_assert(B % NX == 0 && B <= 4, "a tile's chunks stay on fixed buffers");
    auto turn = [&](auto bi) {
      constexpr int b = decltype(bi)::value;
      if constexpr (b < B) {
        compute(buf[b], b % NX, xr[b % NX][0], xr[b % NX][1]);
        issue(buf[b]);
        if constexpr (b % NX == NX - 1) return tile_end();
      }
      return true;
    };
    while (turn(std::integral_constant<int, 0>()) && turn(std::integral_constant<int, 1>()) &&
           turn(std::integral_constant<int, 2>()) && turn(std::integral_constant<int, 3>())) {
    }
  } else {
    int c = 0;
    auto turn = [&](Buf& b) {
      compute(b, c, b.x[0], b.x[1]);
      issue(b);
      if (++c < nc) return true;
      c = 0;
      return tile_end();
    };
    while (turn(buf[0]) && turn(buf[1])) {
    }
  }
  if constexpr (FMT == W_INT4) {
    if (again == 0) return;
    // the lane anew: kept until here it would take a register from the loop
    const int l = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
#pragma unroll 1
    for (q = lo; q < hi; ++q)
#pragma unroll 1
      for (int v = 0; v < VN; ++v) {
        const int64_t col = (int64_t)q * 16 + (l & 15);
        const int t = (l >> 4) + 4 * v;
        if ((q * VN + v) % waves == kp && t < m && col < a.N) int4_redo<G, BF16OUT>(a, sh, t0 + t, col);
      }
  }
}

// 17 to 64 tokens a block.  A wave owns R row tiles over the whole of K, a block of W waves
// 16 R W rows; the tokens pass through LDS in slices of two column steps shared by the
// waves (two buffers: the next slice travels to registers while this one is multiplied,
// one barrier per slice), each fragment read from LDS serving R products.  The codes of
// up to three slices are in flight in registers.
template <int FMT, int G, int R, int W, int NT, bool BF16OUT>
__global__ __launch_bounds__(64 * W) void w4_wide(W4Args a) {
  // Both steps of a slice are multiplied, also where the last has one: the missing one's codes,
  // parameters and tokens are zeros, and without a branch between them the compiler runs the
  // second's loads and products into the first's (N = 12288, K = 4096, 24 tokens: INT4 in
  // groups of 64 20.7 -> 18.2 us, MXFP4 15.5 -> 14.6).  Blocks of 16 row tiles gain nothing
  // or run out of registers (INT4 in groups of 128, N = 65536, 64 tokens: 60 -> 68 us), and so
  // does INT4 in groups of 32 with 64 tokens (42 -> 155).
  constexpr bool BOTH = R == 1 && !(FMT == W_INT4 && G == 32 && NT > 2);
  constexpr int ROWS = 16 * NT, LD = 512 + 16;
  constexpr int PIECES = ROWS * 32 / (64 * W);  // 16-byte pieces of a slice per thread
  __shared__ __attribute__((aligned(16))) uint8_t xs[2][ROWS * LD];
  const int lane = threadIdx.x & 63, g = lane >> 4, wv = uniform(threadIdx.x >> 6);
  const int t0 = blockIdx.y * 64, m = min(ROWS, a.T - t0);
  const W4Shape sh(FMT, a.N, a.K, G);
  const int tiles = (a.N + 15) / 16;
  const int tile0 = (blockIdx.x * W + wv) * R;
  const int slices = (sh.nk + 1) / 2;
  const __amdgpu_buffer_rsrc_t xbuf = make_rsrc(a.x + (size_t)t0 * a.x_ld, ((size_t)(m - 1) * a.x_ld + a.K) * 2);
  int x_off[PIECES], x_lds[PIECES], x_col[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int c = threadIdx.x + i * 64 * W, row = c >> 5, pc = c & 31;
    x_off[i] = min(row, m - 1) * (int)a.x_ld * 2 + pc * 16;
    x_lds[i] = row * LD + pc * 16;
    x_col[i] = pc * 8;
  }
  u32x4 xv[PIECES];
  auto load_slice = [&](int s) {  // columns past K become zeros
#pragma unroll
    for (int i = 0; i < PIECES; ++i) xv[i] = bld16(xbuf, s * 256 + x_col[i] < a.K ? x_off[i] + s * 512 : kPastEnd, 0);
  };
  auto store_slice = [&](int half) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) *reinterpret_cast<u32x4*>(xs[half] + x_lds[i]) = xv[i];
  };
  struct Buf {
    u32x4 w[2][R];
    W4Params<FMT, G> p[R];
  };
  Buf buf[3];
  auto issue = [&](Buf& b, int s) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool tile = tile0 + r < tiles;
      const uint8_t* codes = a.w + (size_t)(tile0 + r) * sh.code_tile;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool live = tile && 2 * s + u < sh.nk;
        b.w[u][r] = bld16(make_rsrc(codes, live ? sh.code_tile : 0), lane * 16, live ? (2 * s + u) * 1024 : 0);
      }
      const bool live = tile && s < slices;
      load_params<FMT, G>(b.p[r], make_rsrc(a.w + sh.par_at + (size_t)(tile0 + r) * sh.par_tile, live ? sh.par_tile : 0),
                          2 * s, live);
    }
  };
  f32x4 acc[R][NT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[r][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Loads return in order, so a slice of tokens is requested ahead of the codes that are
  // needed after it: waiting for slice s + 1 leaves the codes of s + 2 in flight.
  load_slice(0);
  issue(buf[0], 0);
  issue(buf[1], 1);
  store_slice(0);
  load_slice(1);
  issue(buf[2], 2);
  lds_barrier();
  const int row = a_token(lane) * LD;
  int s = 0;
  auto turn = [&](Buf& b) {
    const uint8_t* x = xs[s & 1] + row;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (BOTH || 2 * s + u < sh.nk)
        w4_step<FMT, G, R, NT>(acc, b.w[u], b.p, u, 2 * s + u, [&](int nt, int f) {
          return *reinterpret_cast<const u32x4*>(x + nt * 16 * LD + u * 256 + (FMT == W_MXFP4 ? 64 * g + 16 * f : 64 * f + 16 * g));
        });
    store_slice((s + 1) & 1);
    load_slice(s + 2);  // past the last slice: nothing is read
    issue(b, s + 3);
    lds_barrier();
    return ++s < slices;
  };
  while (turn(buf[0]) && turn(buf[1]) && turn(buf[2])) {
  }
  bool again = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t col = (int64_t)(tile0 + r) * 16 + (lane & 15);
    if (col >= a.N) continue;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int t = nt * 16 + g + 4 * v;
        if (t < m) {
          store_y<BF16OUT>(a, t0 + t, col, acc[r][nt][v]);
          again |= !isfinite(acc[r][nt][v]);
        }
      }
  }
  if constexpr (FMT == W_INT4) {
    if (!again) return;
#pragma unroll 1
    for (int r = 0; r < R; ++r) {
      const int64_t col = (int64_t)(tile0 + r) * 16 + (lane & 15);
#pragma unroll 1
      for (int t = g; t < m && col < a.N; t += 4) int4_redo<G, BF16OUT>(a, sh, t0 + t, col);
    }
  }
}

template <int FMT, int G, bool BF16OUT>
static void launch_t(const W4Args& a, hipStream_t st) {
  const int tiles = (a.N + 15) / 16, pairs = ((a.K + 127) / 128 + 1) / 2;
  if (a.T > 16 && (int64_t)tiles * ((a.T + 15) / 16) >= kW4WideWork) {
    const bool wide = tiles >= (a.T <= 32 ? kW4WideTiles32 : kW4WideTiles);
    const int rows = wide ? 16 : 4;  // row tiles of a block
    const dim3 grid((unsigned)((tiles + rows - 1) / rows), (unsigned)((a.T + 63) / 64));
    if (wide && a.T <= 32) hipLaunchKernelGGL((w4_wide<FMT, G, 2, 8, 2, BF16OUT>), grid, dim3(512), 0, st, a);
    else if (wide) hipLaunchKernelGGL((w4_wide<FMT, G, 2, 8, 4, BF16OUT>), grid, dim3(512), 0, st, a);
    else if (a.T <= 32) hipLaunchKernelGGL((w4_wide<FMT, G, 1, 4, 2, BF16OUT>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((w4_wide<FMT, G, 1, 4, 4, BF16OUT>), grid, dim3(256), 0, st, a);
    return;
  }
  const int nc = (pairs + 15) / 16, waves = (pairs + nc - 1) / nc;
  const int vn = a.T <= 4 ? 1 : a.T <= 8 ? 2 : 4;
  const int per_cu = 16 / waves, fit = 256 * (per_cu > 4 ? 4 : per_cu);
  const dim3 grid((unsigned)(tiles < fit ? tiles : fit), (unsigned)((a.T + 15) / 16)), block(64 * waves);
  const size_t lds = (size_t)2 * vn * waves * 256;
#define MOE_W4_FEW(VN, NC) hipLaunchKernelGGL((w4_few<FMT, G, VN, NC, BF16OUT>), grid, block, lds, st, a, nc)
#define MOE_W4_VN(NC)                \
  do {                               \
    if (vn == 1) MOE_W4_FEW(1, NC);  \
    else if (vn == 2) MOE_W4_FEW(2, NC); \
    else MOE_W4_FEW(4, NC);          \
  } while (0)
  if (nc == 1) MOE_W4_VN(1);
  else if (nc == 2) MOE_W4_VN(2);
  else MOE_W4_VN(0);
#undef MOE_W4_VN
#undef MOE_W4_FEW
}

template <int FMT, int G>
static void launch_out(const W4Args& a, bool bf16_out, hipStream_t st) {
  if (bf16_out) launch_t<FMT, G, true>(a, st);
  else launch_t<FMT, G, false>(a, st);
}

hipError_t launch_w4_linear(int fmt, const W4Args& a, bool bf16_out, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  if (fmt == W_MXFP4) launch_out<W_MXFP4, 32>(a, bf16_out, st);
  else if (a.group == 32) launch_out<W_INT4, 32>(a, bf16_out, st);
  else if (a.group == 64) launch_out<W_INT4, 64>(a, bf16_out, st);
  else launch_out<W_INT4, 128>(a, bf16_out, st);
  return hipGetLastError();
}

}  // namespace moe
